"""Cases of the paged decode operators: what is run, in which form, and what it costs at least.

Four operators around the key scan of a decode step:

* norm_rope  -- RMS norm of each query and key head and the position rotation, in one pass
                (fathom_qk_norm_rope);
* append     -- new keys and values into the pages of a cache, the keys normed and rotated
                on the way (fathom_append_kv);
* attention  -- one query token per sequence over its pages, a prefix that all sequences
                share read once for all (fathom_paged_attention);
* sparse     -- one query token per sequence over the keys its top-k selected, gathered from
                the pages (fathom_sparse_attention_paged).

`own` false computes them with elementary torch operations in 32 bits (angles in 64), true
with the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode token of a Qwen3-8B layer (32 query and 8 KV heads of 128): latency
        {"name": "norm_rope token", "op": "norm_rope", "tokens": 1, "hq": 32, "hkv": 8, "d": 128,
         "dtype": "bf16", "k_dtype": "bf16", "rotary": 128, "interleaved": False,
         "scaling": "none", "factor": 1.0, "norm": True, "far": 131072},
        # an odd chunk of a prompt far into a stretched context: part of a wide head rotated,
        # adjacent pairs, no norm
        {"name": "norm_rope partial far", "op": "norm_rope", "tokens": 4099, "hq": 16, "hkv": 2,
         "d": 256, "dtype": "f16", "k_dtype": "f16", "rotary": 64, "interleaved": True,
         "scaling": "yarn", "factor": 8.0, "norm": False, "far": 1048576},
        # a whole 32k prompt of the layer, the keys widened to float32 for the index
        {"name": "norm_rope prompt 32k", "op": "norm_rope", "tokens": 32768, "hq": 32, "hkv": 8,
         "d": 128, "dtype": "bf16", "k_dtype": "f32", "rotary": 128, "interleaved": False,
         "scaling": "none", "factor": 1.0, "norm": True, "far": 0},
        # one decode step of 16 concurrent sessions
        {"name": "append step of 16", "op": "append", "tokens": 16, "seqs": 16, "hkv": 8,
         "d": 128, "dtype": "bf16", "page": 16, "token_major": False, "rotary": 128,
         "interleaved": False, "scaling": "none", "factor": 1.0, "norm": True, "start": 4096,
         "padded": 0.0},
        # prompts of seven sequences at once, some padding among the tokens
        {"name": "append ragged prompts", "op": "append", "tokens": 20011, "seqs": 7, "hkv": 4,
         "d": 64, "dtype": "f16", "page": 64, "token_major": True, "rotary": 64,
         "interleaved": True, "scaling": "linear", "factor": 4.0, "norm": False, "start": 37,
         "padded": 0.05},
        # a whole 32k prompt of the layer into pages of 32
        {"name": "append prompt 32k", "op": "append", "tokens": 32768, "seqs": 1, "hkv": 8,
         "d": 128, "dtype": "bf16", "page": 32, "token_major": False, "rotary": 128,
         "interleaved": False, "scaling": "none", "factor": 1.0, "norm": True, "start": 0,
         "padded": 0.0},
        # one short session: latency
        {"name": "attention 1 session", "op": "attention", "seqs": 1, "hkv": 8, "group": 4,
         "d": 128, "dtype": "bf16", "page": 16, "token_major": False, "prefix": 0,
         "longest": 2047, "softcap": 0.0, "slopes": False, "empty": False},
        # sessions of uneven length, one of them empty (a padded batch row), capped scores
        {"name": "attention 16 sessions", "op": "attention", "seqs": 16, "hkv": 8, "group": 8,
         "d": 64, "dtype": "f16", "page": 64, "token_major": True, "prefix": 0,
         "longest": 16385, "softcap": 30.0, "slopes": False, "empty": True},
        # agents that share a long system prompt and have their own turns behind it
        {"name": "attention 64 agents 32k", "op": "attention", "seqs": 64, "hkv": 8, "group": 4,
         "d": 128, "dtype": "bf16", "page": 16, "token_major": False, "prefix": 32768,
         "longest": 2048, "softcap": 0.0, "slopes": False, "empty": False},
        # fewer agents, an odd batch and group, scores that fall off with the distance
        {"name": "attention 23 agents biased", "op": "attention", "seqs": 23, "hkv": 4, "group": 5,
         "d": 128, "dtype": "f16", "page": 16, "token_major": False, "prefix": 5008,
         "longest": 301, "softcap": 0.0, "slopes": True, "empty": False},
        # the layer's scan at 131072 keys keeps 2048 per query
        {"name": "sparse 131k top 2048", "op": "sparse", "seqs": 1, "hkv": 8, "group": 4,
         "d": 128, "dtype": "bf16", "page": 16, "token_major": False, "longest": 131072,
         "k": 2048, "softcap": 0.0, "slopes": False, "padded": 0.0},
        # a batch of 16 sessions at top 1024, lists of shorter sessions padded
        {"name": "sparse 16 sessions", "op": "sparse", "seqs": 16, "hkv": 8, "group": 4,
         "d": 128, "dtype": "f16", "page": 32, "token_major": True, "longest": 98304,
         "k": 1024, "softcap": 50.0, "slopes": False, "padded": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "sparse"])
    d = rng.choice([32, 64, 64, 96, 128, 128, 128, 192, 256])
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
    rope = {"rotary": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.4,
            "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
            "norm": rng.random() < 0.6}
    group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8])
    hkv = rng.choice([1, 2, 3, 4, 8])
    kind = {"d": d, "dtype": rng.choice(["bf16", "f16"])}
    pages = {"page": rng.choice([8, 16, 16, 32, 64, 128]), "token_major": rng.random() < 0.4}
    if op == "norm_rope":
        tokens = _log(rng, 1, max(2, 32768 * 5120 // (d * hkv * (group + 3))))
        return {"op": op, "tokens": min(tokens, 32768), "hq": hkv * group, "hkv": hkv, **kind,
                "k_dtype": rng.choice([kind["dtype"], "f32"]), **rope,
                "far": rng.choice([0, 131072, 1048576])}
    if op == "append":
        seqs = _log(rng, 1, 64)
        tokens = min(32768, 32768 * 1024 // (d * hkv))
        return {"op": op, "tokens": max(seqs, _log(rng, 1, tokens)), "seqs": seqs, "hkv": hkv,
                **kind, **pages, **rope, "start": _log(rng, 1, 4096),
                "padded": rng.choice([0.0, 0.0, 0.05])}
    scores = {"softcap": rng.choice([0.0, 0.0, 20.0, 50.0]), "slopes": rng.random() < 0.3}
    if op == "attention":
        room = 163840 * 1024 // (d * hkv)          # keys that the largest listed case holds
        seqs = _log(rng, 1, 64)
        # and the products that it makes over its prefix
        most = min(32768, room // 2, (1 << 33) // (d * hkv * group * seqs))
        prefix = _log(rng, 64, most) // pages["page"] * pages["page"] if rng.random() < 0.6 else 0
        longest = _log(rng, 1, max(2, min(32768, (room - prefix) // seqs)))
        return {"op": op, "seqs": seqs, "hkv": hkv, "group": group, **kind, **pages,
                "prefix": prefix, "longest": longest, **scores, "empty": rng.random() < 0.2}
    seqs = _log(rng, 1, 16)
    longest = _log(rng, 64, min(131072, (1 << 31) // (d * hkv * seqs)))
    return {"op": op, "seqs": seqs, "hkv": hkv, "group": group, **kind, **pages,
            "longest": longest, "k": _log(rng, 1, min(2048, longest)), **scores,
            "padded": rng.choice([0.0, 0.1])}


# ------------------------------------------------------------------------------ inputs
def _lens(case):
    """Keys that each sequence has of its own: uneven, one at the full length, one empty if asked."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["longest"], case.get("k", 0)))
    lens = [rng.randint(max(1, case["longest"] // 2), case["longest"]) for _ in range(case["seqs"])]
    lens[0] = case["longest"]
    if case.get("empty") and len(lens) > 1:
        lens[-1] = 0
    return lens


def _frequencies(case, device):
    """Radians per position of each rotated pair (float64), and the magnitude of the rotation."""
    rd, s, base, original = case["rotary"], case["factor"], 1e6, 32768
    if case["scaling"] == "ntk" and rd > 2:
        base = base * s ** (rd / (rd - 2))
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=device) / rd)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "yarn":
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * keep + f / s * (1 - keep), 0.1 * math.log(s) + 1.0
    return f, 1.0


def _rotary(case):
    import decode_fathom_plan_b200 as fp
    return fp.RotaryTable(case["d"], case["rotary"], base=1e6, interleaved=case["interleaved"],
                          scaling=case["scaling"], factor=case["factor"], original_len=32768,
                          beta_fast=32.0, beta_slow=1.0)


def _channels(shape, gen, dtype, d):
    """Rows whose channels have lognormal scales, a few of them ten times as large."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    sigma = torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    sigma[torch.randperm(d, generator=gen, device="cuda")[:max(1, d // 32)]] *= 10
    return x.mul_(sigma.to(dtype))


def _pool(n_pages, case, gen):
    shape = [n_pages, case["hkv"], case["page"], case["d"]]
    if case["token_major"]:
        shape[1], shape[2] = shape[2], shape[1]
    k = _channels(shape, gen, DTYPES[case["dtype"]], case["d"])
    v = torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[case["dtype"]])
    return (k.transpose(1, 2), v.transpose(1, 2)) if case["token_major"] else (k, v)


def _table(counts, shared, gen):
    """Page table [seqs][most] of scattered pages, the first `shared` the same in every row,
    -1 behind a row's last page; and the pages of the pool."""
    total = shared + sum(counts)
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), shared + max(counts + [1])), -1, dtype=torch.int32, device="cuda")
    table[:, :shared] = perm[:shared]
    at = shared
    for b, n in enumerate(counts):
        table[b, shared:shared + n] = perm[at:at + n]
        at += n
    return table, max(1, total)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    op, d, dt = case["op"], case["d"], DTYPES[case["dtype"]]
    if op in ("norm_rope", "append"):
        T, hkv, hq = case["tokens"], case["hkv"], case.get("hq", 0)
        # rows of the projection: queries, keys and values of a token side by side
        qkv = _channels([T, hq + 2 * hkv, d], gen, dt, d)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        w = 1 + 0.2 * torch.randn([2, d], generator=gen, device="cuda")
        st["q_weight"], st["k_weight"] = w.to(dt) if case["norm"] else (None, None)
        st["freq"], st["mag"] = _frequencies(case, "cuda")
        if own:
            st["table"] = _rotary(case)
    if op == "norm_rope":
        st["pos"] = (case["far"] + torch.arange(T, device="cuda")).to(torch.int32)
        st["q_out"] = torch.empty([T, hq, d], dtype=dt, device="cuda")
        k_out = torch.empty([hkv, T, d], dtype=DTYPES[case["k_dtype"]], device="cuda")
        st["k_out"] = k_out.transpose(0, 1)
    elif op == "append":
        n = case["seqs"]
        seq = (torch.arange(T, device="cuda") * n // T).to(torch.int32)
        first = torch.searchsorted(seq, torch.arange(n, device="cuda", dtype=torch.int32))
        starts = torch.randint(0, case["start"] + 1, [n], generator=gen, device="cuda")
        st["pos"] = (torch.arange(T, device="cuda") - first[seq.long()] + starts[seq.long()]).to(torch.int32)
        if case["padded"]:
            seq[torch.rand(T, generator=gen, device="cuda") < case["padded"]] = -1
        st["seq"] = seq
        pages = -(-(case["start"] + -(-T // n) + 1) // case["page"])
        st["pages"], total = _table([pages] * n, 0, gen)
        st["ck"], st["cv"] = _pool(total, case, gen)
        if own:
            import decode_fathom_plan_b200 as fp
            st["cache"] = fp.PagedKV.from_tensors(st["ck"], st["cv"])
    else:
        lens, page = _lens(case), case["page"]
        shared = case.get("prefix", 0)
        st["pages"], total = _table([-(-n // page) for n in lens], shared // page, gen)
        st["ck"], st["cv"] = _pool(total, case, gen)
        hq = case["hkv"] * case["group"]
        st["q"] = torch.randn([len(lens), hq, d], generator=gen, device="cuda", dtype=dt)
        full = [n + shared if n else 0 for n in lens]
        st["max_len"] = max(full)
        st["lens"] = torch.tensor(full, dtype=torch.int32, device="cuda")
        st["scale"] = 1.0 / math.sqrt(d)
        st["slopes"] = None
        if case["slopes"]:
            st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float32, device="cuda") / hq)
        st["out"] = torch.empty_like(st["q"])
        if op == "sparse":
            k = case["k"]
            # k distinct keys of each sequence, ascending: one from each of k equal runs; a
            # list longer than its sequence, and a share of the rest, is padded with -1
            u = torch.rand([len(lens), hq, k], generator=gen, device="cuda", dtype=torch.float64)
            n = st["lens"].double()[:, None, None]
            i = torch.arange(k, device="cuda", dtype=torch.float64)
            run = torch.clamp(n / k, min=1.0)
            j = torch.floor(torch.ceil(i * run) + u * (torch.ceil((i + 1) * run) - torch.ceil(i * run)))
            j[j >= n] = -1
            if case["padded"]:
                j[torch.rand(j.shape, generator=gen, device="cuda") < case["padded"]] = -1
            st["idx"] = j.to(torch.int32)
        if own:
            import decode_fathom_plan_b200 as fp
            st["cache"] = fp.PagedKV.from_tensors(st["ck"], st["cv"])
            if op == "sparse":
                ws = fp.fathom_sparse_attention_paged_workspace_bytes(len(lens), hq, d, case["k"])
            else:
                ws = fp.fathom_paged_attention_workspace_bytes(st["cache"].desc, len(lens), case["group"],
                                                               st["max_len"], shared)
            st["workspace"] = torch.empty(max(16, ws), dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------------------- plain forms
def _plain_norm_rope(x, weight, pos, st):
    """float32 [T][h][d]: norm of each head, then the rotation of its first channels."""
    case = st["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rd = case["rotary"]
    angle = pos.double()[:, None] * st["freq"]
    cos = (angle.cos() * st["mag"]).float()[:, None]
    sin = (angle.sin() * st["mag"]).float()[:, None]
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if case["interleaved"] else (x[..., :rd // 2], x[..., rd // 2:rd])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if case["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rd:]], -1)


def _plain_append(st):
    case = st["case"]
    keep = st["seq"] >= 0
    seq, pos = st["seq"][keep].long(), st["pos"][keep]
    page = st["pages"][seq, (pos // case["page"]).long()].long()
    at = (pos % case["page"]).long()
    k = _plain_norm_rope(st["k"][keep], st["k_weight"], pos, st)
    st["ck"][page, :, at] = k.to(st["ck"].dtype)
    st["cv"][page, :, at] = st["v"][keep].to(st["cv"].dtype)
    return st["ck"], st["cv"]


def _softmax_parts(logits, seen):
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top.masked_fill(torch.isinf(top), 0.0))
    return p, p.sum(-1, keepdim=True)


def _logits(dots, st, distance):
    """Capped and biased logits from dots [..., hkv, g, n] and distances that broadcast to them."""
    case = st["case"]
    s = dots * st["scale"]
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    if st["slopes"] is not None:
        s = s - st["slopes"].view(case["hkv"], case["group"], 1) * distance
    return s


def _plain_attention(st):
    case = st["case"]
    B, H, G, d = case["seqs"], case["hkv"], case["group"], case["d"]
    n_pre = case["prefix"] // case["page"]
    q = st["q"].float().view(B, H, G, d)
    lens = st["lens"].long()
    # the shared prefix once, [H][prefix][d]; each sequence's own keys padded, [B][H][longest][d]
    first = st["pages"][0, :n_pre].long()
    pk, pv = (c[first].float().transpose(0, 1).reshape(H, -1, d) for c in (st["ck"], st["cv"]))
    rest = st["pages"][:, n_pre:].clamp(min=0).long()
    sk, sv = (c[rest].float().transpose(1, 2).reshape(B, H, -1, d) for c in (st["ck"], st["cv"]))
    dots = torch.cat([torch.einsum("bhgd,hnd->bhgn", q, pk), q @ sk.transpose(-1, -2)], -1)
    j = torch.arange(dots.shape[-1], device=q.device)
    seen = (j < lens[:, None])[:, None, None]
    p, total = _softmax_parts(_logits(dots, st, (lens[:, None] - 1 - j)[:, None, None].float()), seen)
    out = torch.einsum("bhgn,hnd->bhgd", p[..., :case["prefix"]], pv) + p[..., case["prefix"]:] @ sv
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.view(B, H * G, d).to(st["q"].dtype)


def _plain_sparse(st):
    case = st["case"]
    B, H, G, d, k = case["seqs"], case["hkv"], case["group"], case["d"], case["k"]
    idx = st["idx"].view(B, H, G, k)
    seen, j = idx >= 0, idx.clamp(min=0).long()
    page = torch.gather(st["pages"][:, None, None].expand(B, H, G, -1), 3, j // case["page"]).long()
    head = torch.arange(H, device=j.device)[:, None, None]
    kr = st["ck"][page, head, j % case["page"]].float()
    vr = st["cv"][page, head, j % case["page"]].float()
    dots = (kr @ st["q"].float().view(B, H, G, d, 1)).squeeze(-1)
    far = st["lens"].long()[:, None, None, None] - 1 - j
    p, total = _softmax_parts(_logits(dots, st, far.float()), seen)
    out = (p.unsqueeze(-2) @ vr).squeeze(-2)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.view(B, H * G, d).to(st["q"].dtype)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import decode_fathom_plan_b200 as fp
        if op == "norm_rope":
            fp.fathom_qk_norm_rope(st["q"], st["k"], st["pos"], st["q_out"], st["k_out"], rotary=st["table"],
                                   q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS)
            return st["q_out"], st["k_out"]
        if op == "append":
            fp.fathom_append_kv(st["cache"].desc, st["k"], st["v"], st["seq"], st["pos"], st["pages"],
                                rotary=st["table"], k_weight=st["k_weight"], eps=EPS)
            return st["ck"], st["cv"]
        if op == "attention":
            fp.fathom_paged_attention(st["cache"].desc, st["q"], st["pages"], st["lens"], st["max_len"],
                                      st["out"], st["workspace"], st["scale"], prefix_len=case["prefix"],
                                      softcap=case["softcap"], slopes=st["slopes"])
            return st["out"]
        fp.fathom_sparse_attention_paged(st["cache"].desc, st["q"], st["idx"], st["pages"], st["lens"],
                                         st["out"], st["workspace"], st["scale"],
                                         softcap=case["softcap"], slopes=st["slopes"])
        return st["out"]
    if op == "norm_rope":
        q = _plain_norm_rope(st["q"], st["q_weight"], st["pos"], st)
        k = _plain_norm_rope(st["k"], st["k_weight"], st["pos"], st)
        return q.to(st["q_out"].dtype), k.to(st["k_out"].dtype)
    if op == "append":
        return _plain_append(st)
    return _plain_attention(st) if op == "attention" else _plain_sparse(st)


# ---------------------------------------------------------------------------- the floor
def work(case):
    op, d = case["op"], case["d"]
    if op == "norm_rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        out = 4 if case["k_dtype"] == "f32" else 2
        return {"bytes": t * d * (4 * hq + (2 + out) * hkv) + 4 * t, "flops": t * (hq + hkv) * (6 * d)}
    if op == "append":
        t = int(case["tokens"] * (1 - case["padded"]))
        return {"bytes": t * case["hkv"] * d * 8 + 12 * case["tokens"], "flops": t * case["hkv"] * 6 * d}
    lens, h, g = _lens(case), case["hkv"], case["group"]
    rows = 4 * case["seqs"] * h * g * d            # the queries and the outputs
    if op == "attention":
        keys = case["prefix"] + sum(lens)
        pairs = sum(n + case["prefix"] for n in lens if n)
        return {"bytes": 4 * keys * h * d + rows + 4 * keys // case["page"], "flops": 4 * pairs * h * g * d}
    share = 1 - case["padded"]
    took = [min(case["k"], n) * share for n in lens]
    # rows of a KV head that at least one of its g queries selected
    rows_read = sum(h * n * (1 - (1 - t / n) ** g) for t, n in zip(took, lens))
    return {"bytes": 4 * rows_read * d + rows + 4 * case["seqs"] * h * g * case["k"],
            "flops": 4 * sum(took) * h * g * d}


# ------------------------------------------------------------------------------- oracle
def _exact_turn(x, weight, pos, st):
    """64 bits: each pair of channels as a complex number times magnitude * e^(i angle)."""
    case = st["case"]
    y = x.to(torch.float64)
    if weight is not None:
        rms = torch.sqrt((y * y).sum(-1) / y.shape[-1] + EPS)
        y = y / rms.unsqueeze(-1) * weight.to(torch.float64)
    half = case["rotary"] // 2
    unit = torch.arange(half, device=x.device)
    lo, hi = (2 * unit, 2 * unit + 1) if case["interleaved"] else (unit, unit + half)
    z = torch.complex(y[..., lo], y[..., hi])
    angle = pos.to(torch.float64).view(-1, 1, 1) * st["freq"].view(1, 1, -1)
    z = z * torch.polar(torch.full_like(angle, float(st["mag"])), angle)
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_row(st, q, keys, values, j, length, heads):
    """One sequence's query heads [h][d] over the rows keys, values [h][n][d] of positions j."""
    case = st["case"]
    s = (keys * q.to(torch.float64).unsqueeze(1)).sum(-1) * st["scale"]
    if case["softcap"]:
        s = torch.tanh(s / case["softcap"]) * case["softcap"]
    if st["slopes"] is not None:
        s = s - st["slopes"][heads].to(torch.float64).unsqueeze(1) * (length - 1 - j)
    return (torch.softmax(s, -1).unsqueeze(-1) * values).sum(1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return tuple(_exact_turn(st[n], st[n + "_weight"], st["pos"], st) for n in ("q", "k"))
    page = case["page"]
    if op == "append":
        seq, pos = st["seq"].cpu().numpy(), st["pos"].cpu().numpy()
        table = st["pages"].cpu().numpy()
        live = np.flatnonzero(seq >= 0)
        row = torch.from_numpy(table[seq[live], pos[live] // page].astype(np.int64)).cuda()
        col = torch.from_numpy((pos[live] % page).astype(np.int64)).cuda()
        tok = torch.from_numpy(live).cuda()
        ck, cv = st["ck"].to(torch.float64), st["cv"].to(torch.float64)
        turned = _exact_turn(st["k"][tok], st["k_weight"], st["pos"][tok], st)
        for h in range(case["hkv"]):
            ck[row, h, col] = turned[:, h]
            cv[row, h, col] = st["v"][tok, h].to(torch.float64)
        return ck, cv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    g = case["group"]
    for b, n in enumerate(st["lens"].tolist()):
        if op == "attention":
            if not n:
                continue
            j = torch.arange(n, device="cuda")
            pg = st["pages"][b].long()[j // page]
            for h in range(case["hkv"]):
                heads = torch.arange(h * g, h * g + g, device="cuda")
                keys = st["ck"][pg, h, j % page].to(torch.float64)
                values = st["cv"][pg, h, j % page].to(torch.float64)
                for i in range(g):
                    out[b, h * g + i] = _exact_row(st, st["q"][b, h * g + i][None], keys[None], values[None],
                                                   j, n, heads[i:i + 1])[0]
        else:
            for i in range(case["hkv"] * g):
                j = st["idx"][b, i].long()
                j = j[j >= 0]
                if j.numel():
                    pg = st["pages"][b].long()[j // page]
                    keys = st["ck"][pg, i // g, j % page].to(torch.float64)
                    values = st["cv"][pg, i // g, j % page].to(torch.float64)
                    out[b, i] = _exact_row(st, st["q"][b, i][None], keys[None], values[None], j, n,
                                           torch.tensor([i], device="cuda"))[0]
    return out
