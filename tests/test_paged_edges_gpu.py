"""Calls on a paged cache at the edges of what their documentation allows: padded batch rows before
the others, waits that run out, probabilities far below the largest, sizes past 32 bits."""
import math

import numpy as np
import pytest
import torch

import decode_fathom_plan_b200 as fp
from tests import paged_oracle as po
from tests.test_paged_edges_cpu import yarn_index
from tests.test_paged_gpu import BF16, F16, Batch, check, check_rows, few_rows, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp.load_library()
    torch.cuda.set_device(0)
    fp.fathom_last_device_status()


# ------------------------------------------------- a shared prefix behind padded batch rows
def shared(lens, dtype=BF16, prefix=2048, H=8, G=2, d=64, page=16, seed=50):
    """A batch whose repeated reads of the prefix pass the 8 MB from which one kernel serves them all."""
    assert 4 * d * H * prefix * (len(lens) - 1) >= 8 << 20
    return Batch(lens, prefix, H, G, d, page, dtype, False, seed)


@pytest.mark.parametrize("first", [1, 2, 37])
@pytest.mark.parametrize("entry", [-7, 0, 5, 2 ** 31 - 1])
def test_prefix_of_a_batch_whose_first_rows_are_padded(first, entry):
    """An empty sequence's row of the table holds anything; the prefix is read by another's."""
    b = shared([0] * first + [2100, 0, 2049, 2048])
    b.table_t[:first] = entry
    b.attention()
    assert status() == fp.FATHOM_OK
    assert (b.out[:first] == 0).all() and (b.out[first + 1] == 0).all()
    check_rows(b, {(s, i) for s in (0, first, first + 2, first + 3) for i in (0, 7, 15)})
    one = b.out.clone()
    b.prefix = 0                                    # each sequence reads the prefix for itself
    b.attention()
    assert status() == fp.FATHOM_OK
    check_rows(b, {(s, i) for s in (0, first, first + 2, first + 3) for i in (0, 7, 15)})
    assert (one[:first] == 0).all()


@pytest.mark.parametrize("length", [-1, 5, 10 ** 6])
def test_prefix_is_not_read_by_the_row_of_a_refused_length(length):
    b = shared([2060, 2100, 2049, 2050, 2051])
    b.lens_t[0] = length
    b.table_t[0] = 3
    b.attention()
    assert status() == fp.FATHOM_ERR_INVALID_ARG
    assert (b.out[0] == 0).all()
    check_rows(b, {(s, i) for s in range(1, 5) for i in (0, 9, 15)})


def test_prefix_of_a_batch_of_padded_rows_alone():
    b = shared([2060, 2100, 2049, 2050, 2051])
    b.lens_t.zero_()
    b.table_t.fill_(-9)
    b.attention()
    assert status() == fp.FATHOM_OK                 # no entry of the table was used
    assert (b.out == 0).all()


# ---------------------------------------------------------------------- waits that run out
@pytest.fixture
def limit():
    before = fp.fathom_set_wait_limit(500000000)
    assert before == 500000000
    yield fp.fathom_set_wait_limit
    fp.fathom_set_wait_limit(before)


WAITS = [
    # lens, H, G, d, dtype: two row blocks, the even and odd tiles of one, one slot
    ([2048 + 37 * (i % 4) for i in range(40)], 2, 4, 128, BF16),
    ([4096 + 5 * i for i in range(5)], 4, 3, 64, F16),
    ([2048, 0, 2100, 2300], 4, 8, 256, BF16),
]


@pytest.mark.parametrize("lens,H,G,d,dtype", WAITS)
def test_a_wait_that_runs_out_is_reported_and_joins_nothing_unwritten(lens, H, G, d, dtype, limit):
    prefix = lens[0]
    b = shared(lens, dtype, prefix, H, G, d)
    b.attention()
    assert status() == fp.FATHOM_OK
    whole = b.out.clone()
    # no wait is over at its first look: what is left are the keys behind the prefix
    limit(0)
    b.ws.fill_(0xFF)                                # parts that nobody writes are NaN
    b.attention(ws=b.ws)
    assert status() == fp.FATHOM_ERR_TIMEOUT and status() == fp.FATHOM_OK
    own = np.full((len(lens), H * G, max(lens) - prefix), -1)
    for s, n in enumerate(lens):
        own[s, :, :max(0, n - prefix)] = np.arange(prefix, max(n, prefix))
    want, tol = b.expect(idx=own)
    check(b.out, want, tol)
    # limits that run out with copies and products under way
    for ns in (200, 1000, 3000, 6000, 12000, 25000):
        limit(ns)
        for _ in range(3):
            b.ws.fill_(0xFF)
            b.attention(ws=b.ws)
            assert status() in (fp.FATHOM_OK, fp.FATHOM_ERR_TIMEOUT)
            assert torch.isfinite(b.out).all()
    limit(500000000)
    b.attention(ws=b.ws)
    assert status() == fp.FATHOM_OK and torch.equal(b.out, whole)


# ------------------------------------------------ one workspace while sessions come and go
def test_one_workspace_for_the_largest_batch_and_every_smaller_one():
    G, d, prefix = 4, 128, 2048
    b = shared([prefix + 9 * i for i in range(40)], BF16, prefix, 8, G, d)
    longest = max(b.lens)
    need = fp.fathom_paged_attention_workspace_bytes(b.kv.desc, 40, G, longest, prefix)
    hq, k = 8 * G, 600
    idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(40, hq, 1)
    need_sparse = fp.fathom_sparse_attention_paged_workspace_bytes(40, hq, d, k)
    guard, guard_sparse = (torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
                           for n in (need, need_sparse))
    q, out, table, lens_t, lens = b.q, b.out, b.table_t, b.lens_t, b.lens
    for n in (40, 33, 32, 21, 2, 1):
        b.lens, b.lens_t, b.table_t = lens[:n], lens_t[:n], table[:n]
        b.q, b.out = q[:n], out[:n]
        b.attention(max_len=longest, ws=guard[:need])
        check_rows(b, {(0, 0), (n - 1, hq - 1), (n // 2, 5)})
        fp.fathom_sparse_attention_paged(b.kv.desc, b.q, idx[:n], b.table_t, b.lens_t, b.out,
                                         guard_sparse[:need_sparse], b.scale)
        at = {(0, 0), (n - 1, hq - 1), (n // 2, 5)}
        want, tol = b.expect(idx=idx[:n].cpu().numpy(), rows=at, round_p=False)
        rows = tuple(np.array(sorted(at)).T)
        check(b.out.cpu()[rows], want[rows], tol[rows])
    assert status() == fp.FATHOM_OK
    assert (guard[need:] == 0xA5).all() and (guard_sparse[need_sparse:] == 0xA5).all()


# ------------------------------------------------- one key that outweighs a long tail of others
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,prefix,H", [([1024] * 8, 0, 32), ([516, 515], 512, 75)])
@pytest.mark.parametrize("nats", [8.0, 13.0, 16.0, 17.2, 17.4])
def test_a_key_far_above_the_others_leaves_them_their_weight(lens, prefix, H, dtype, nats):
    """A key whose value is zero takes nearly all of the weight; what is left are the others.

    A float16 probability is a multiple of 2^-24 at least, half a step 2^-25, of a scale 2^7 times
    that of the reference maximum, which is at most the row's maximum: 2^-32 of the largest weight.
    At 17.2 nats a key weighs 2^-24.8 of it, so its rounding is 2^-7.2 of it, and that of all of
    them 1 in 140 of the result, whatever their number."""
    d = 64
    b = Batch(lens, prefix, H, 1, d, 16, dtype, False, 5)
    assert not prefix or 4 * d * H * prefix * (len(lens) - 1) >= 8 << 20
    k, v = torch.zeros_like(b.kv.k), (64 * (1 + b.kv.v * 0.1)).to(dtype)
    for s in range(len(lens)):
        k[b.table[s, 0], :, 0, 0], v[b.table[s, 0], :, 0] = nats, 0.0
    b.kv.k.copy_(k)
    b.kv.v.copy_(v)
    b.k64, b.v64 = po.f64(b.kv.k), po.f64(b.kv.v)
    b.q.zero_()
    b.q[:, :, 0] = 8.0                                      # times 1/sqrt(64): a score is the key's first channel
    b.attention()
    assert status() == fp.FATHOM_OK
    q, step, tiny = po.f64(b.q), po.HALF_STEP[dtype], po.TINY[dtype]
    for s, i in ((0, 0), (len(lens) - 1, H - 1), (1, H // 2)):
        ks, vs = (po.gather(p, b.table[s], np.arange(lens[s]), i, 16) for p in (b.k64, b.v64))
        want, err = po.attend(q[s, i], ks, vs, np.zeros(lens[s]), b.scale, p_step=step, p_tiny=tiny * 2.0 ** -7)
        check(b.out[s, i], want, err + step * np.abs(want) * 1.01 + tiny, (s, i))


def test_rows_turned_by_yarn_over_pair_numbers():
    T, h, d = 37, 3, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn([T, h, d], generator=g).to(BF16).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 5003
    out = torch.empty([T, h, d], dtype=torch.float32, device="cuda")
    tab = fp.RotaryTable(d, base=1e6, scaling="yarn_index", factor=8.0, original_len=32768)
    fp.fathom_qk_norm_rope(x, None, pos, out, None, tab)
    freq, _, _ = yarn_index(d, 1e6, 8.0, 32768, 32.0, 1.0)
    y, size = po.norm_rope(po.f64(x), pos.cpu().numpy().astype(np.float64), None, 1e-6, freq,
                           0.1 * math.log(8.0) + 1.0)
    check(out, y, po.norm_rope_tolerance(y, size, torch.float32))


@pytest.mark.parametrize("rd,inter", [(64, False), (48, True), (2, False)])
def test_rows_turned_by_given_frequencies(rd, inter):
    T, h, d = 9, 2, 64
    g = torch.Generator().manual_seed(rd)
    x = torch.randn([T, h, d], generator=g).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1009
    freq = torch.rand([rd // 2], generator=g, dtype=torch.float64) * 3 - 1      # any, negative ones too
    tab = fp.RotaryTable.from_frequencies(freq, d, inter, 1.25)
    out = torch.empty_like(x)
    fp.fathom_qk_norm_rope(x, None, pos, out, None, tab)
    y, size = po.norm_rope(po.f64(x), pos.cpu().numpy().astype(np.float64), None, 1e-6, freq.numpy(), 1.25, inter)
    check(out, y, po.norm_rope_tolerance(y, size, torch.float32))
    same = fp.RotaryTable(d, rd, 1e4, inter)
    again = fp.RotaryTable.from_frequencies([1e4 ** (-2 * i / rd) for i in range(rd // 2)], d, inter)
    assert torch.allclose(same.turns, again.turns, rtol=1e-14, atol=0)


# ------------------------------------------------------------- bfloat16 probabilities in two terms
@pytest.mark.parametrize("lens", [[16], [1024, 48], [700]])
@pytest.mark.parametrize("G,d", [(4, 128), (8, 64), (1, 96), (3, 256)])
def test_bfloat16_probabilities_of_own_keys_keep_sixteen_bits(lens, G, d):
    """Of every 16 keys one has the largest weight, 1, and 15 a weight that bfloat16 rounds badly;
    their values all but cancel, so that the rounding of the output hides nothing.

    What one term leaves of a weight is at most 2^-8 of it, what the second leaves of that 2^-16."""
    H, page = 2, 16
    b = Batch(lens, 0, H, G, d, page, BF16, False, 3)
    scores = torch.arange(-256, 0).to(BF16).unique()[:-1] / 64
    weights = torch.exp(scores.double())
    off = (weights.float().to(BF16).double() - weights).abs() / weights
    at = int(off.argmax())
    weight = float(weights[at])
    top = float(torch.tensor(-15 * weight).to(BF16))            # value of the largest, against 15 ones
    k, v = torch.zeros_like(b.kv.k), torch.ones_like(b.kv.v)
    k[..., 0] = float(scores[at])
    k[:, :, 5, 0] = 0.0                                         # one slot of each page of 16
    v[:, :, 5] = top
    b.kv.k.copy_(k)
    b.kv.v.copy_(v)
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.scale = 1.0
    b.attention()
    assert status() == fp.FATHOM_OK
    for s, n in enumerate(lens):
        j = np.arange(n)
        ks, vs = np.zeros((n, d)), np.ones((n, d))
        ks[:, 0] = np.where(j % page == 5, 0.0, float(scores[at]))
        vs[j % page == 5] = top
        want, err = po.attend(po.f64(b.q)[s, 0], ks, vs, np.zeros(n), 1.0, p_step=2.0 ** -16)
        tol = err + po.HALF_STEP[BF16] * np.abs(want) * 1.01
        # a weight in one term alone would be seen
        p = np.exp(ks[:, 0])
        one = torch.from_numpy(p).float().to(BF16).double().numpy() @ vs / p.sum()
        assert (np.abs(one - want) > 4 * tol).all()
        for i in range(H * G):
            check(b.out[s, i], want, tol, (s, i))


# --------------------------------------------------- sums that nothing but the inputs decides
@pytest.mark.parametrize("G,d,dtype", [(3, 128, BF16), (5, 128, BF16), (6, 64, F16), (7, 256, BF16), (5, 192, F16)])
def test_sums_do_not_depend_on_what_ran_before(G, d, dtype):
    """A slot of 128 rows holds 128 / G whole sequences; behind them lies what another kernel left in
    shared memory, which must not decide when the other rows of a warp renew their maximum."""
    prefix, H = 2048, 2
    bs = [shared([prefix + 40 + i for i in range(2 * (128 // G) + 3)], dtype, prefix, H, G, d, seed=60 + i)
          for i in range(2)]
    bs[1].q.mul_(40)                                            # leaves large rows behind
    bs[1].kv.k.mul_(4)
    want = None
    for _ in range(12):
        for b in bs:
            b.attention(ws=getattr(b, "ws", None))
        want = bs[0].out.clone() if want is None else want
        assert torch.equal(bs[0].out, want)
        bs[0].out.fill_(math.nan)
        torch.cuda.synchronize()
        bs[0].attention(ws=bs[0].ws)
        assert torch.equal(bs[0].out, want)
    assert status() == fp.FATHOM_OK
    check_rows(bs[0], few_rows(bs[0], 4))


# ------------------------------------------------------------------ calls that follow one another
@pytest.mark.parametrize("lens,H,G,d", [([2048 + 40 + 11 * i for i in range(9)], 8, 4, 64),
                                        ([1024 + 600 + i for i in range(33)], 2, 5, 128)])
def test_attention_reads_what_the_call_before_it_wrote(lens, H, G, d):
    """The kernel of the own keys starts beside that of the prefix: keys, lengths and pages that were
    written just before are the new ones, with and without a wait of the host in between."""
    n, prefix = len(lens), lens[0] // 1024 * 1024
    b = shared(lens, BF16, prefix, H, G, d)
    g = torch.Generator(device="cuda").manual_seed(4)
    ks = torch.randn([40, n, H, d], generator=g, device="cuda").to(BF16)
    qs = torch.randn([40, n, H * G, d], generator=g, device="cuda").to(BF16)
    seq = torch.arange(n, dtype=torch.int32, device="cuda")
    full, table = b.lens_t.clone(), b.table_t.clone()
    b.attention()

    start = b.kv.k.clone(), b.kv.v.clone()

    def steps(wait):
        outs = []
        b.kv.k.copy_(start[0])
        b.kv.v.copy_(start[1])
        for i in range(40):
            pos = full - 1 - i % 7
            fp.fathom_append_kv(b.kv.desc, ks[i], ks[39 - i], seq, pos, table)
            if wait:
                torch.cuda.synchronize()
            b.q = qs[i]
            torch.add(pos, 1, out=b.lens_t)                     # a kernel of another library before the call
            b.attention(max_len=max(lens), ws=b.ws)
            fp.fathom_append_kv(b.kv.desc, ks[39 - i], ks[i], seq, pos, table)   # and one that overwrites after it
            b.attention(max_len=max(lens), ws=b.ws)
            outs.append(b.out.clone())
            if wait:
                torch.cuda.synchronize()
        return torch.stack(outs)

    first = steps(True)
    for _ in range(5):
        assert torch.equal(steps(False), first)
    assert status() == fp.FATHOM_OK


def test_the_whole_step_captured_and_replayed():
    """Norm, rotation, append, plan, scan, and both attentions as one graph."""
    H, G, d, page, n, k = 2, 4, 128, 16, 4000, 256
    hq = H * G
    g = torch.Generator(device="cuda").manual_seed(9)
    kv = fp.PagedKV(n // page + 2, page, H, d)
    kv.k.copy_(torch.randn(kv.k.shape, generator=g, device="cuda"))
    kv.v.copy_(torch.randn(kv.v.shape, generator=g, device="cuda"))
    table = torch.randperm(n // page + 1, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    ix = fp.KeyIndex(H, G, n, d)
    ix.pack(torch.randn([H, n, d], generator=g, device="cuda"))
    buf = fp.ScanBuffers(ix, k)
    rot = fp.RotaryTable(d, base=1e6)
    w = torch.ones(d, dtype=BF16, device="cuda")
    qkv = torch.empty([1, hq + 2 * H, d], dtype=BF16, device="cuda")
    pos, lens, seq = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3))
    q = torch.empty([1, hq, d], dtype=BF16, device="cuda")
    k32 = torch.empty([1, H, d], device="cuda")
    some, every = torch.empty_like(q), torch.empty_like(q)
    budget = torch.full([hq], 2 * d, dtype=torch.int32, device="cuda")
    ws, ws2 = (torch.empty(1 << 22, dtype=torch.uint8, device="cuda") for _ in range(2))

    def step():
        fp.fathom_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + H], pos, q, k32, rot, w, w)
        fp.fathom_append_kv(kv.desc, qkv[:, hq:hq + H], qkv[:, hq + H:], seq, pos, table, rot, w)
        fp.plan_and_scan(ix, q.view(hq, d).view(torch.int16), budget, buf)
        fp.fathom_sparse_attention_paged(kv.desc, q, buf.idx[None], table, lens, some, ws, d ** -0.5)
        fp.fathom_paged_attention(kv.desc, q, table, lens, n + page, every, ws2, d ** -0.5)

    def inputs(i):
        qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda"))
        pos.fill_(n - 20 + i)
        lens.fill_(n - 19 + i)

    inputs(0)
    lens.fill_(n)
    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.capture_begin()
        step()
        graph.capture_end()
    for i in range(6):
        inputs(i)
        lens.fill_(n)
        for out in (some, every, q, k32):
            out.fill_(math.nan)
        step()
        want = [x.clone() for x in (q, k32, some, every, kv.k, buf.idx)]
        for out in (some, every, q, k32):
            out.fill_(math.nan)
        graph.replay()
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip((q, k32, some, every, kv.k, buf.idx), want))
        assert torch.isfinite(some).all() and torch.isfinite(every).all()
    assert status() == fp.FATHOM_OK


# ------------------------------------------------------------- layouts and sizes at their ends
@pytest.mark.parametrize("prefix", [0, 2048])
@pytest.mark.parametrize("q_heads_first,out_heads_first", [(False, True), (True, False)])
@pytest.mark.parametrize("G,d,dtype", [(4, 128, BF16), (3, 96, F16), (1, 256, BF16)])
def test_attention_on_views(prefix, q_heads_first, out_heads_first, G, d, dtype):
    """Queries inside a projection or stored head by head, outputs likewise, keys and values of several
    layers side by side in one pool."""
    H, page, lens = 4, 16, [prefix + 5, 0, prefix + 77, prefix + 1, prefix + 16] + [prefix + 30] * 9
    b = Batch(lens, prefix, H, G, d, page, dtype, False, 70)
    n, hq = len(lens), H * G
    pool = torch.full([b.kv.k.shape[0], 3, page, 2, H, d + 32], math.nan, dtype=dtype, device="cuda")
    k, v = (pool[:, 1, :, i, :, :d].transpose(1, 2) for i in range(2))
    k.copy_(b.kv.k)
    v.copy_(b.kv.v)
    b.kv = fp.PagedKV.from_tensors(k, v)

    def rows(heads_first):
        if heads_first:
            return torch.full([hq + 1, n, d], math.nan, dtype=dtype, device="cuda")[1:].transpose(0, 1)
        return torch.full([n, hq + 2 * H, d + 8], math.nan, dtype=dtype, device="cuda")[:, 1:1 + hq, :d]
    q, out = rows(q_heads_first), rows(out_heads_first)
    q.copy_(b.q)
    b.q, b.out = q, out
    b.attention()
    assert status() == fp.FATHOM_OK
    at = {(s, i) for s in (0, 1, 2, n - 1) for i in (0, hq - 1)}
    check_rows(b, at)
    idx = np.full((n, hq, 40), -1, np.int32)
    for s, m in enumerate(lens):
        if m:
            idx[s] = np.random.default_rng(s).integers(0, m, (hq, 40))
    ws = torch.empty(max(16, fp.fathom_sparse_attention_paged_workspace_bytes(n, hq, d, 40)), dtype=torch.uint8,
                     device="cuda")
    fp.fathom_sparse_attention_paged(b.kv.desc, b.q, torch.from_numpy(idx).cuda(), b.table_t, b.lens_t, b.out, ws,
                                     b.scale)
    want, tol = b.expect(idx=idx, rows=at, round_p=False)
    where = tuple(np.array(sorted(at)).T)
    check(b.out.cpu()[where], want[where], tol[where])


@pytest.mark.parametrize("n,H,G,prefix", [(65535, 1, 1, 0), (65535, 1, 1, 8), (3001, 2, 5, 64), (2, 700, 8, 512)])
def test_largest_batches_and_most_heads(n, H, G, prefix):
    d, page = 32, 8
    rng = np.random.default_rng(n)
    lens = [int(x) for x in np.where(rng.random(n) < 0.2, 0, prefix + rng.integers(1, 20, n))]
    lens[-1] = prefix + 19
    b = Batch(lens, prefix, H, G, d, page, BF16, False, 71)
    b.attention()
    assert status() == fp.FATHOM_OK
    hq = H * G
    at = {(int(s), int(i)) for s, i in zip(rng.integers(0, n, 40), rng.integers(0, hq, 40))} | {(0, 0), (n - 1, hq - 1)}
    check_rows(b, at)
    empty = torch.tensor(lens, device="cuda") == 0
    assert (b.out[empty] == 0).all()
    k = 5
    idx = np.where(np.array(lens)[:, None, None] > 0, rng.integers(0, np.maximum(lens, 1)[:, None, None], (n, hq, k)),
                   -1).astype(np.int32)
    ws = torch.empty(fp.fathom_sparse_attention_paged_workspace_bytes(n, hq, d, k), dtype=torch.uint8, device="cuda")
    b.out.fill_(math.nan)
    fp.fathom_sparse_attention_paged(b.kv.desc, b.q, torch.from_numpy(idx).cuda(), b.table_t, b.lens_t, b.out, ws,
                                     b.scale)
    want, tol = b.expect(idx=idx, rows=at, round_p=False)
    where = tuple(np.array(sorted(at)).T)
    check(b.out.cpu()[where], want[where], tol[where])
    assert status() == fp.FATHOM_OK and (b.out[empty] == 0).all()


def test_a_sequence_of_more_keys_than_a_float_counts():
    """17 million keys, 8 queries, a bias by distance; the same keys selected by a list of their ends."""
    n, G, d, page = (1 << 24) + 300001, 8, 32, 1024
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(2)
    kv = fp.PagedKV(pages, page, 1, d)
    for x in (kv.k, kv.v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda", dtype=BF16))
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    q = torch.randn([1, G, d], generator=g, device="cuda").to(BF16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    slopes = torch.tensor([0.0, 0.0, 1e-6, 1e-5, 1e-4, 0.01, 1.0, 0.0], device="cuda")
    ws = torch.empty(fp.fathom_paged_attention_workspace_bytes(kv.desc, 1, G, n), dtype=torch.uint8, device="cuda")
    fp.fathom_paged_attention(kv.desc, q, table, lens, n, out, ws, d ** -0.5, slopes=slopes)
    assert status() == fp.FATHOM_OK
    j = torch.arange(n, device="cuda")
    at = table[0].long()[j // page] * page + j % page
    keys, values = (x.reshape(-1, d)[at].double() for x in (kv.k, kv.v))
    dist = (n - 1 - j).double()
    for i in range(G):
        s = keys @ q[0, i].double() * d ** -0.5 - slopes[i].double() * dist
        p = torch.exp(s - s.max())
        want, size = p @ values / p.sum(), p @ values.abs() / p.sum()
        # scores of up to 6 and biases, each to 2^-17 and 2^-21 of itself where the weight is (within 20
        # of the largest), two-term probabilities, the rounding of the output
        tol = size * (6 * 2.0 ** -17 + 2.0 ** -19 + 2.0 ** -16 + 26 * 2.0 ** -21) + want.abs() * 2.0 ** -8
        check(out[0, i], want.cpu().numpy(), tol.cpu().numpy(), i)


def test_rows_whose_offsets_pass_32_bits():
    T, h, d, far = 4, 2, 64, 1 << 30
    pool = torch.empty(3 * far + h * d, dtype=BF16, device="cuda")
    x = pool.as_strided([T, h, d], [far, d, 1])
    g = torch.Generator().manual_seed(3)
    src = torch.randn([T, h, d], generator=g).to(BF16)
    w = (1 + torch.rand([d], generator=g)).to(BF16).cuda()
    pos = torch.tensor([5, 2 ** 20, 0, 77], dtype=torch.int32, device="cuda")
    tab = fp.RotaryTable(d, base=1e6)
    y, size = po.norm_rope(po.f64(src), pos.cpu().numpy().astype(np.float64), po.f64(w), 1e-6, po.turns(d, 1e6)[0])
    tol = po.norm_rope_tolerance(y, size, BF16)
    x.copy_(src)
    near = torch.empty([T, h, d], dtype=BF16, device="cuda")
    fp.fathom_qk_norm_rope(x, None, pos, near, None, tab, w)
    check(near, y, tol)
    fp.fathom_qk_norm_rope(None, x, pos, None, x, tab, None, w)             # in place, far apart
    check(x, y, tol)
    x.copy_(src)
    kv = fp.PagedKV(2, 8, h, d)
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    slot = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    fp.fathom_append_kv(kv.desc, x, x, seq, slot, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), None, w)
    y, size = po.norm_rope(po.f64(src), None, po.f64(w))
    for t in range(T):
        at = int(slot[t])
        check(kv.k[1 - at // 8, :, at % 8], y[t], po.norm_rope_tolerance(y, size, BF16)[t])
        assert torch.equal(kv.v[1 - at // 8, :, at % 8].cpu(), src[t])
    assert status() == fp.FATHOM_OK


@pytest.mark.parametrize("T,hq,hk,d,dtype", [(1, 65535, 1, 32, BF16), (3, 1, 4097, 96, F16), (70001, 1, 1, 32, BF16)])
def test_norm_rope_of_most_heads_and_tokens(T, hq, hk, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k = (torch.randn([T, n, d], generator=g, device="cuda").to(dtype) for n in (hq, hk))
    w = (1 + torch.rand([d], generator=g, device="cuda")).to(dtype)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 11
    q_out, k_out = torch.full_like(q, math.nan), torch.full([T, hk, d], math.nan, device="cuda")
    fp.fathom_qk_norm_rope(q, k, pos, q_out, k_out, fp.RotaryTable(d, base=1e5), w, None)
    p = pos.cpu().numpy().astype(np.float64)
    for x, out, weight in ((q, q_out, w), (k, k_out, None)):
        y, size = po.norm_rope(po.f64(x), p, None if weight is None else po.f64(weight), 1e-6, po.turns(d, 1e5)[0])
        check(out, y, po.norm_rope_tolerance(y, size, out.dtype))
    assert status() == fp.FATHOM_OK
