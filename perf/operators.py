"""The cache operators of this library as measured cases: block means of the
keys, the selection of kv blocks by a block score, and attention of a few
query tokens per sequence (one token, a draft chain or a draft tree) over a
contiguous or paged cache, dense or over selected blocks.

``run`` with ``own`` false computes them in elementary torch operations;
with ``own`` true it makes the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_NONE = 0xFFFF  # unused index slot


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the prompt of a batch has been written to its pages: means of every block
        dict(name="means_prompt", op="means", layout="PA_BBND", B=8, N2=8, D=128, lo=8192, hi=32768,
             page=128, BKV=128, append=0, dtype="bf16"),
        # one token was appended to every sequence: only its last block changes
        dict(name="means_append", op="means", layout="PA_BBND", B=64, N2=8, D=128, lo=1000, hi=16384,
             page=256, BKV=128, append=1, dtype="bf16"),
        # packed training sequences of odd lengths, wide blocks, small heads
        dict(name="means_packed", op="means", layout="TND", B=5, N2=6, D=64, lo=333, hi=9001,
             page=0, BKV=512, append=0, dtype="fp16"),
        # block index of a long causal prompt, one row per query head
        dict(name="select_prompt", op="select", layout="BNSD", B=1, N1=24, N2=24, D=128, T=32768,
             lo=32768, hi=32768, BQ=128, BKV=128, W=16, rows="query", causal=True, sink=1, local=1,
             dtype="bf16"),
        # ragged packed prompts, the heads of a group share their row
        dict(name="select_ragged", op="select", layout="TND", B=8, N1=32, N2=8, D=128, T=0, lo=512,
             hi=4096, BQ=128, BKV=128, W=8, rows="group", causal=False, sink=0, local=1, dtype="fp16"),
        # one new token per sequence chooses among the blocks of a long cache
        dict(name="select_decode", op="select", layout="TND", B=64, N1=32, N2=8, D=128, T=1, lo=4096,
             hi=131072, BQ=128, BKV=128, W=64, rows="group", causal=False, sink=1, local=2,
             dtype="bf16"),
        # the smallest call: one sequence, one token, a short cache
        dict(name="decode_one", op="decode", layout="PA_BBND", B=1, T=1, N1=32, N2=8, D=128, lo=1024,
             hi=1024, page=128, BKV=128, W=0, rows="group", mask="none", dtype="bf16"),
        # a serving batch over the blocks that it selected
        dict(name="decode_sparse", op="decode", layout="PA_BBND", B=32, T=1, N1=32, N2=8, D=128,
             lo=8192, hi=32768, page=128, BKV=128, W=32, rows="group", mask="none", dtype="bf16"),
        # a serving batch over its whole caches, the largest read
        dict(name="decode_dense", op="decode", layout="PA_BBND", B=16, T=1, N1=64, N2=8, D=128,
             lo=4097, hi=65536, page=256, BKV=128, W=0, rows="group", mask="none", dtype="fp16"),
        # a small draft tree of one sequence, contiguous cache, small heads
        dict(name="tree_small", op="decode", layout="BNSD", B=1, T=24, N1=16, N2=4, D=64, lo=1500,
             hi=1500, page=0, BKV=128, W=0, rows="group", mask="tree", dtype="bf16"),
        # draft trees of a serving batch
        dict(name="tree_batch", op="decode", layout="PA_BBND", B=16, T=32, N1=32, N2=8, D=128, lo=2048,
             hi=16384, page=128, BKV=128, W=0, rows="group", mask="tree", dtype="bf16"),
        # wide draft trees, more than one mask word and several row tiles
        dict(name="tree_wide", op="decode", layout="PA_BBND", B=4, T=96, N1=32, N2=4, D=128, lo=16384,
             hi=32768, page=128, BKV=128, W=0, rows="group", mask="tree", dtype="fp16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["means", "select", "decode", "decode"])
    dtype = rng.choice(["bf16", "fp16"])
    D = rng.choice([64, 128, 128])
    BKV = rng.choice([128, 128, 256, 512])
    page = rng.choice([128, 256, 512])
    if op == "means":
        layout = rng.choice(["PA_BBND", "PA_BBND", "TND", "BNSD"])
        B, N2 = _log(rng, 1, 32), rng.choice([1, 2, 3, 8])
        hi = max(64, min(_log(rng, 64, 65536), 160000 * 8 // (B * N2)))
        return dict(op=op, layout=layout, B=B, N2=N2, D=D, lo=rng.randint(1, hi), hi=hi,
                    page=page, BKV=BKV, append=rng.choice([0, 0, 1, 5]), dtype=dtype)
    g = rng.choice([1, 2, 3, 4, 6, 8])
    if op == "select":
        N2 = rng.choice([1, 2, 4, 8])
        if rng.random() < 0.5:  # one or a few new tokens per sequence
            B, T = _log(rng, 1, 64), rng.choice([1, 1, 2, 7])
            hi = _log(rng, 64 * BKV, 131072)
            lo = rng.randint(hi // 4, hi)
            causal = False
        else:  # a prompt
            BKV = min(BKV, 256)
            hi = _log(rng, 4000, 16384)
            B, T, lo = rng.randint(1, max(1, min(8, 32768 // hi))), 0, rng.randint(hi // 2, hi)
            causal = rng.choice([True, True, False])
        # fewer than the blocks of the shortest sequence, more than the forced ones
        W = rng.choice([w for w in (4, 5, 8, 13, 32, 64) if w == 4 or 4 * w < 3 * (lo // BKV)])
        return dict(op=op, layout="TND", B=B, N1=g * N2, N2=N2, D=D, T=T, lo=lo, hi=hi,
                    BQ=rng.choice([128, 256]), BKV=BKV, W=W,
                    rows=rng.choice(["group", "query"]), causal=causal, sink=rng.choice([0, 1]),
                    local=rng.choice([0, 1]), dtype=dtype)
    N2 = rng.choice([1, 2, 3, 8])
    layout = rng.choice(["PA_BBND", "PA_BBND", "BNSD"])
    mask = rng.choice(["none", "none", "tree", "causal"])
    T = 1 if mask == "none" else rng.choice([2, 5, 8, 16, 33, 64, 100])
    hi = max(300, _log(rng, 300, 32768))
    B = _log(rng, 1, max(1, min(64, 2000000 // (hi * N2 * max(1, T * g // 64)))))
    W = rng.choice([0, 0, 3, 16, 40])
    return dict(op=op, layout=layout, B=B, T=T, N1=g * N2, N2=N2, D=D, lo=rng.randint(max(T, hi // 6), hi),
                hi=hi, page=page, BKV=BKV, W=W, rows=rng.choice(["group", "query"]) if W else "group",
                mask=mask, dtype=dtype)


def _lens(case):
    """The kv lengths of the batch: spread over [lo, hi], the longest first."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    return [hi - int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(B)]


def _nb(case):
    return max(-(-n // case["BKV"]) for n in _lens(case))


# ------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, dtype, g):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=g)


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int64, device="cuda")


def _cache(case, names, g, extra=None):
    """Key (and value) caches in the case's layout, and the tensors that say
    where a sequence's tokens are."""
    lens, B, N2, D, dt = _lens(case), case["B"], case["N2"], case["D"], _DT[case["dtype"]]
    s = {}
    if case["layout"] == "PA_BBND":
        page = case["page"]
        most = max(-(-n // page) for n in lens)
        total = sum(-(-n // page) for n in lens) + 3
        for n in names:
            s[n] = _normal((total, page, N2, D), dt, g)
        perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
        table, at = torch.zeros(B, most, dtype=torch.int32), 0
        perm = perm.cpu()
        for b, n in enumerate(lens):
            k = -(-n // page)
            table[b, :k] = perm[at:at + k]
            at += k
        s["table"] = table.cuda()
        s["used"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    elif case["layout"] == "TND":
        for n in names:
            s[n] = _normal((sum(lens), N2, D), dt, g)
        s["cu_kv"] = _cu(lens)
    else:
        for n in names:
            s[n] = _normal((B, N2, max(lens), D), dt, g)
        s["used"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return s


def _trees(B, T, seed):
    """Ancestor bits of random trees: node j sees itself and its ancestors."""
    words = -(-T // 64)
    rng = random.Random(seed)
    out = []
    for _ in range(B):
        bits = []
        for j in range(T):
            up = 0 if j == 0 else bits[rng.randrange(max(0, j - 12), j)]
            bits.append(up | (1 << j))
        for m in bits:
            for w in range(words):
                x = (m >> (64 * w)) & ((1 << 64) - 1)
                out.append(x - (1 << 64) if x >> 63 else x)
    return torch.tensor(out, dtype=torch.int64).view(B, T, words).cuda()


def _rows_plan(case):
    """Packed prompts: the sequence and query block of every token and row."""
    q_lens = _lens(case) if case["T"] == 0 else [case["T"]] * case["B"]
    row_of, row_b, last = [], [], []
    for b, n in enumerate(q_lens):
        for i in range(-(-n // case["BQ"])):
            rows = min(case["BQ"], n - i * case["BQ"])
            row_of += [len(row_b)] * rows
            row_b.append(b)
            last.append(i * case["BQ"] + rows - 1 - n)  # relative to the end of the sequence
    return q_lens, row_of, row_b, last


def prepare(case, seed):
    g = _gen(seed)
    dt, B, N2, D = _DT[case["dtype"]], case["B"], case["N2"], case["D"]
    s = dict(case=case)
    if case["op"] == "means":
        s |= _cache(case, ["k"], g)
        # an append works on means that are there; a prompt fills a fresh buffer
        s["means"] = _normal((B, N2, _nb(case), D), dt, g) if case["append"] else \
            torch.zeros(B, N2, _nb(case), D, dtype=dt, device="cuda")
        lens = torch.tensor(_lens(case), device="cuda")
        if case["append"]:
            s["first"] = (lens - case["append"]).clamp(min=0).to(torch.int32)
    elif case["op"] == "select":
        N1, BKV = case["N1"], case["BKV"]
        lens = _lens(case)
        # keys share a direction within a block more than across the cache
        s["means"] = (0.25 * _normal((B, N2, _nb(case), D), torch.float32, g)).to(dt)
        s["used"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if case["layout"] == "BNSD":
            s["q"] = _normal((B, N1, case["T"], D), dt, g)
        else:
            q_lens, row_of, row_b, last = _rows_plan(case)
            s["q"] = _normal((sum(q_lens), N1, D), dt, g)
            s["cu_q"], s["cu_kv"] = _cu(q_lens), _cu(lens)
            s["row_of"] = torch.tensor(row_of, device="cuda")
            s["row_b"] = torch.tensor(row_b, device="cuda")
            s["last"] = torch.tensor(last, device="cuda")
    else:
        N1, T = case["N1"], case["T"]
        s |= _cache(case, ["k", "v"], g)
        lens = torch.tensor(_lens(case), device="cuda")
        s["q"] = _normal((B, N1, T, D) if case["layout"] == "BNSD" else (B * T, N1, D), dt, g)
        if case["layout"] == "PA_BBND":
            s["cu_q"] = _cu([T] * B)
        if case["mask"] == "tree":
            s["tree"] = _trees(B, T, seed)
            if case["layout"] == "PA_BBND":
                s["tree"] = s["tree"].view(B * T, -1)
        if case["W"]:
            # every row keeps its last block and random others, ascending
            H = N1 if case["rows"] == "query" else N2
            nb = _nb(case)
            nk = (lens + case["BKV"] - 1) // case["BKV"]
            r = torch.rand(B, H, nb, device="cuda", generator=g)
            ids = torch.arange(nb, device="cuda")
            r = torch.where(ids == (nk - 1).view(B, 1, 1), 2.0, r)
            r = torch.where(ids < nk.view(B, 1, 1), r, -1.0)
            W = min(case["W"], nb)
            val, top = r.topk(W, dim=-1)
            top = torch.where(val >= 0, top, _NONE).sort(-1).values
            if W < case["W"]:
                top = torch.nn.functional.pad(top, (0, case["W"] - W), value=_NONE)
            rows = -(-T // 128)  # every query block of a sequence has a row of its own
            top = top.unsqueeze(2).expand(B, H, rows, case["W"])
            if case["layout"] == "PA_BBND":
                top = top.transpose(0, 1).reshape(H, B * rows, case["W"])
            s["index"] = top.contiguous().to(torch.int32).to(torch.uint16)
    return s


# --------------------------------------------------------------------- plain
def _tokens(s, name, at):
    """Rows `at` [B, n] (token numbers) of a cache, [B, n, N2, D]."""
    c, x = s["case"], s[name]
    b = torch.arange(c["B"], device="cuda").view(-1, 1)
    if c["layout"] == "PA_BBND":
        page = s["table"].long()[b, at // c["page"]]
        return x[page, at % c["page"]]
    if c["layout"] == "TND":
        return x[s["cu_kv"][:-1].view(-1, 1) + at]
    return x[b, :, at]


def _kv_lens(s):
    return s["used"].long() if "used" in s else s["cu_kv"][1:] - s["cu_kv"][:-1]


def _plain_means(s):
    c = s["case"]
    lens, BKV, B, nb = _kv_lens(s), c["BKV"], c["B"], s["means"].shape[2]
    if not c["append"]:
        u = torch.arange(nb * BKV, device="cuda").expand(B, -1)
        real = u < lens.view(-1, 1)
        k = _tokens(s, "k", torch.where(real, u, 0)).float() * real.view(B, -1, 1, 1)
        n = (lens.view(-1, 1) - torch.arange(nb, device="cuda") * BKV).clamp(0, BKV)
        m = k.view(B, nb, BKV, c["N2"], c["D"]).sum(2) / n.clamp(min=1).view(B, nb, 1, 1)
        m = m.transpose(1, 2).to(s["means"].dtype)
        s["means"].copy_(torch.where((n > 0).view(B, 1, nb, 1), m, s["means"]))
        return s["means"]
    # the blocks from the first new token's to the last: at most `span` of them
    span = (c["append"] + BKV - 2) // BKV + 1
    blk = (s["first"].long() // BKV).view(-1, 1) + torch.arange(span, device="cuda")
    u = (blk.unsqueeze(-1) * BKV + torch.arange(BKV, device="cuda"))
    real = u < lens.view(-1, 1, 1)
    k = _tokens(s, "k", torch.where(real, u, 0).view(B, -1)).float() * real.view(B, -1, 1, 1)
    n = real.sum(-1)
    m = k.view(B, span, BKV, c["N2"], c["D"]).sum(2) / n.clamp(min=1).view(B, span, 1, 1)
    # blocks past the last are written over the last one's own value
    keep = (n > 0).long().cumsum(1).argmax(1, keepdim=True)
    to = torch.where(n > 0, torch.arange(span, device="cuda"), keep)
    b = torch.arange(B, device="cuda").view(-1, 1)
    s["means"].transpose(1, 2)[b, blk.gather(1, to)] = m[b, to].to(s["means"].dtype)
    return s["means"]


def _plain_select(s):
    c = s["case"]
    B, N1, N2, D, BKV, W = c["B"], c["N1"], c["N2"], c["D"], c["BKV"], c["W"]
    lens, nb = _kv_lens(s), s["means"].shape[2]
    m = s["means"].double()
    if c["layout"] == "BNSD":
        T, BQ = c["T"], c["BQ"]
        R = -(-T // BQ)
        q = torch.nn.functional.pad(s["q"], (0, 0, 0, R * BQ - T)).double()
        q = q.view(B, N1, R, BQ, D).sum(3)  # [B, N1, R, D]
        if c["rows"] == "group":
            q = q.view(B, N2, N1 // N2, R, D).sum(2)
        sc = torch.matmul(q.view(B, N2, -1, D), m.transpose(2, 3)).view(B, -1, R, nb)
        end = (torch.arange(1, R + 1, device="cuda") * BQ).clamp(max=T) - 1 - T
        end = end.view(1, 1, R) + lens.view(B, 1, 1)  # the last kv token that a block's last row sees
        lens = lens.view(B, 1, 1)
    else:
        R = s["row_b"].shape[0]
        q = torch.zeros(R, N1, D, dtype=torch.float64, device="cuda").index_add_(0, s["row_of"], s["q"].double())
        if c["rows"] == "group":
            q = q.view(R, N2, N1 // N2, D).sum(2)
        mr = m[s["row_b"]]  # [R, N2, nb, D]
        sc = torch.matmul(q.view(R, N2, -1, D), mr.transpose(2, 3)).view(R, -1, nb).transpose(0, 1)
        end = (lens[s["row_b"]] + s["last"]).view(1, R)
        lens = lens[s["row_b"]].view(1, R)
    nk = (lens + BKV - 1) // BKV
    if c["causal"]:
        nk = torch.minimum(nk, torch.div(end, BKV, rounding_mode="floor") + 1).clamp(min=0)
    ids, nk = torch.arange(nb, device="cuda"), nk.unsqueeze(-1)
    can = ids < nk
    must = can & ((ids < c["sink"]) | (ids >= nk - c["local"]))
    sc = torch.where(must, math.inf, torch.where(can, sc, -math.inf))
    top = torch.sort(sc, dim=-1, descending=True, stable=True).indices[..., :W]
    got = torch.where(can.expand(sc.shape).gather(-1, top), top, _NONE).sort(-1).values
    if W > nb:
        got = torch.nn.functional.pad(got, (0, W - nb), value=_NONE)
    return got.to(torch.int32).to(torch.uint16)


def _plain_decode(s):
    c = s["case"]
    B, T, N1, N2, D, W = c["B"], c["T"], c["N1"], c["N2"], c["D"], c["W"]
    g, lens = N1 // N2, _kv_lens(s)
    q = s["q"].float()
    q = q if c["layout"] == "BNSD" else q.view(B, T, N1, D).transpose(1, 2)  # [B, N1, T, D]
    q = q.reshape(B, N2, g, T, D)
    if W:  # one key list per row of the index
        ix = s["index"].to(torch.int32).long()
        if c["layout"] == "PA_BBND":
            ix = ix.view(ix.shape[0], B, -1, W).transpose(0, 1)
        ix = ix[:, :, 0]  # the query blocks of a sequence carry the same row
        H = ix.shape[1]
        u = (ix.unsqueeze(-1) * c["BKV"] + torch.arange(c["BKV"], device="cuda")).view(B, H, -1)
        real = (ix != _NONE).repeat_interleave(c["BKV"], -1) & (u < lens.view(B, 1, 1))
        u = torch.where(real, u, 0)
        b = torch.arange(B, device="cuda").view(B, 1, 1)
        h = (torch.arange(H, device="cuda") * N2 // H).view(1, H, 1)
        if c["layout"] == "PA_BBND":
            at = (s["table"].long()[b, u // c["page"]], u % c["page"], h)
        else:
            at = (b, h, u)
        k, v = s["k"][at].float(), s["v"][at].float()  # [B, H, n, D]
        k, v = k.view(B, N2, H // N2, -1, D), v.view(B, N2, H // N2, -1, D)
        u, real = u.view(B, N2, H // N2, 1, -1), real.view(B, N2, H // N2, 1, -1)
    else:
        n = max(_lens(c))
        if c["layout"] == "BNSD":
            k, v = s["k"].float().unsqueeze(2), s["v"].float().unsqueeze(2)
        else:
            at = torch.arange(n, device="cuda").expand(B, -1)
            at = torch.where(at < lens.view(-1, 1), at, 0)
            k = _tokens(s, "k", at).float().transpose(1, 2).unsqueeze(2)
            v = _tokens(s, "v", at).float().transpose(1, 2).unsqueeze(2)
        u = torch.arange(n, device="cuda").view(1, 1, 1, 1, -1)
        real = u < lens.view(B, 1, 1, 1, 1)
    if not W or c["rows"] == "group":
        q = q.reshape(B, N2, 1, g * T, D)  # rows that share their keys
    sc = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    node = u - (lens.view(B, 1, 1, 1, 1) - T)  # draft node of a key; negative: context
    if c["mask"] == "tree":
        bits = s["tree"].view(B, 1, 1, T, -1)
        j = node.clamp(0, T - 1)
        word = bits.expand(B, j.shape[1], j.shape[2], T, bits.shape[-1]).gather(
            -1, (j // 64).expand(B, j.shape[1], j.shape[2], T, j.shape[-1]))
        see = (node < 0) | (((word >> (j % 64)) & 1) != 0)
    elif c["mask"] == "causal":
        see = node <= torch.arange(T, device="cuda").view(1, 1, 1, T, 1)
    else:
        see = node < T
    see = see & real
    if q.shape[3] != see.shape[3] and see.shape[3] != 1:
        see = see.repeat(1, 1, 1, g, 1)
    sc = sc.masked_fill(~see, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(sc - top)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    lse = (top + torch.log(l)).view(B, N1, T)
    o = o.view(B, N1, T, D).to(s["q"].dtype)
    if c["layout"] == "BNSD":
        return o, lse
    return o.transpose(1, 2).reshape(B * T, N1, D), lse.transpose(1, 2).reshape(B * T, N1)


# ----------------------------------------------------------------------- own
def _own(s):
    import block_sparse_variable_b200 as bsa
    c = s["case"]
    lay, ws = c["layout"], s.get("ws")
    if c["op"] == "means":
        P = bsa.params_for("BNSD" if lay == "BNSD" else "TND", lay, c["N2"], c["N2"], (128, c["BKV"]))
        means, s["ws"] = bsa.bsa_block_means(s["k"], P, cu_seqlens_kv=s.get("cu_kv"),
                                             seqused_kv=s.get("used"), block_table=s.get("table"),
                                             first_kv=s.get("first"), means=s["means"], workspace=ws)
        return means
    if c["op"] == "select":
        P = bsa.params_for(lay, lay, c["N1"], c["N2"], (c["BQ"], c["BKV"]), causal=c["causal"])
        rows = -(-c["T"] // c["BQ"]) if lay == "BNSD" else s["row_b"].shape[0]
        index, s["ws"] = bsa.bsa_select_blocks(
            s["q"], s["means"], P, width=c["W"], index_heads=c["N1"] if c["rows"] == "query" else c["N2"],
            rows=rows, sink_blocks=c["sink"], local_blocks=c["local"], cu_seqlens_q=s.get("cu_q"),
            cu_seqlens_kv=s.get("cu_kv"), seqused_kv=s["used"], workspace=ws)
        return index
    P = bsa.params_for("BNSD" if lay == "BNSD" else "TND", lay, c["N1"], c["N2"], (128, c["BKV"]),
                       causal=c["mask"] == "causal")
    out, lse, s["ws"] = bsa.bsa_decode(s["q"], s["k"], s["v"], P, index=s.get("index"),
                                       tree_mask=s.get("tree"), cu_seqlens_q=s.get("cu_q"),
                                       seqused_kv=s.get("used"), block_table=s.get("table"),
                                       workspace=ws)
    return out, lse


def run(state):
    if own:
        return _own(state)
    return {"means": _plain_means, "select": _plain_select, "decode": _plain_decode}[state["case"]["op"]](state)


# ----------------------------------------------------------------------- work
def work(case):
    lens, N2, D, BKV = _lens(case), case["N2"], case["D"], case["BKV"]
    row = N2 * D * 2
    if case["op"] == "means":
        if case["append"]:
            first = [max(0, n - case["append"]) // BKV for n in lens]
            toks = sum(n - f * BKV for n, f in zip(lens, first))
            blocks = sum(-(-n // BKV) - f for n, f in zip(lens, first))
        else:
            toks, blocks = sum(lens), sum(-(-n // BKV) for n in lens)
        return {"bytes": (toks + blocks) * row, "flops": toks * N2 * D}
    N1 = case["N1"]
    if case["op"] == "select":
        H = N1 if case["rows"] == "query" else N2
        q_lens = lens if case["layout"] == "TND" and case["T"] == 0 else [case["T"]] * case["B"]
        pairs = rows = 0
        for n, t in zip(lens, q_lens):
            nk, nq = -(-n // BKV), -(-t // case["BQ"])
            rows += nq
            for i in range(nq):
                last = min(t, (i + 1) * case["BQ"]) - 1 + n - t
                pairs += min(nk, last // BKV + 1) if case["causal"] else nk
        toks = sum(q_lens)
        return {"bytes": toks * N1 * D * 2 + sum(-(-n // BKV) for n in lens) * row + H * rows * case["W"] * 2,
                "flops": toks * N1 * D + 2 * D * pairs * H}
    T, g, toks, pairs = case["T"], N1 // N2, 0.0, 0.0
    for n in lens:
        nk = -(-n // BKV)
        w = min(case["W"], nk) if case["W"] else nk
        mine = min(n, w * BKV) if case["W"] else n
        pairs += mine * T * N1
        if case["W"] and case["rows"] == "query":  # blocks that any head of the group keeps, in the mean
            mine = n * (1.0 - (1.0 - w / nk) ** g)
        toks += mine
    q = case["B"] * T * N1
    return {"bytes": 2 * toks * row + q * (2 * D * 2 + 4), "flops": 4 * D * pairs}


# ---------------------------------------------------------------------- exact
def _one_sequence(s, name, b, n):
    """The n tokens of sequence b in 64 bits, [N2, n, D]."""
    c, x = s["case"], s[name]
    if c["layout"] == "PA_BBND":
        pages = s["table"][b, :-(-n // c["page"])].long()
        return x[pages].flatten(0, 1)[:n].double().transpose(0, 1)
    if c["layout"] == "TND":
        at = sum(_lens(c)[:b])
        return x[at:at + n].double().transpose(0, 1)
    return x[b, :, :n].double()


def _exact_means(s):
    c, BKV = s["case"], s["case"]["BKV"]
    out = s["means"].double()
    for b, n in enumerate(_lens(c)):
        k = _one_sequence(s, "k", b, n)
        first = max(0, n - c["append"]) // BKV if c["append"] else 0
        for j in range(first, -(-n // BKV)):
            out[b, :, j] = k[:, j * BKV:min(n, (j + 1) * BKV)].mean(1)
    return out


def _exact_select(s):
    c = s["case"]
    BQ, BKV, W, g = c["BQ"], c["BKV"], c["W"], c["N1"] // c["N2"]
    group, at, cols = c["rows"] == "group", 0, []
    for b, n in enumerate(_lens(c)):
        t = c["T"] or n
        q = s["q"][b].double() if c["layout"] == "BNSD" else s["q"][at:at + t].double().transpose(0, 1)
        at += t
        m = s["means"][b].double().repeat_interleave(1 if group else g, 0)  # [H, nb, D]
        for i in range(-(-t // BQ)):
            x = q[:, i * BQ:(i + 1) * BQ]
            end = i * BQ + x.shape[1] - 1 + n - t
            nk = -(-n // BKV)
            if c["causal"]:
                nk = max(0, min(nk, end // BKV + 1))
            x = x.sum(1)
            if group:
                x = x.view(-1, g, x.shape[-1]).sum(1)
            sc = (m[:, :nk] * x.unsqueeze(1)).sum(-1)
            sc[:, :c["sink"]] = math.inf
            if c["local"]:
                sc[:, max(0, nk - c["local"]):] = math.inf
            ahead = (sc.unsqueeze(1) > sc.unsqueeze(2)).sum(-1)
            same = (sc.unsqueeze(1) == sc.unsqueeze(2)).tril(-1).sum(-1)
            pick = ahead + same < W
            row = torch.full((sc.shape[0], W), _NONE, device="cuda")
            for h, ids in enumerate(pick):
                ids = ids.nonzero().view(-1)
                row[h, :ids.numel()] = ids
            cols.append(row)
    out = torch.stack(cols, 1)  # [H, rows of the batch, W]
    if c["layout"] == "BNSD":
        out = out.view(out.shape[0], c["B"], -1, W).transpose(0, 1)
    return out.to(torch.int32).to(torch.uint16)


def _exact_decode(s):
    c = s["case"]
    T, N1, N2, D, W = c["T"], c["N1"], c["N2"], c["D"], c["W"]
    g = N1 // N2
    outs, lses = [], []
    for b, n in enumerate(_lens(c)):
        k, v = _one_sequence(s, "k", b, n), _one_sequence(s, "v", b, n)
        see = torch.ones(T, n, dtype=torch.bool, device="cuda")
        if c["mask"] == "causal":
            see = torch.ones(T, n, dtype=torch.bool, device="cuda").tril(n - T)
        elif c["mask"] == "tree":
            w = s["tree"][b] if c["layout"] == "BNSD" else s["tree"][b * T:(b + 1) * T]
            for j in range(T):
                see[:, n - T + j] = ((w[:, j // 64] >> (j % 64)) & 1).bool()
        oo, ll = [], []
        for h in range(N1):
            ok = see
            if W:
                hi = h if c["rows"] == "query" else h // g
                row = s["index"].to(torch.int32)
                row = row[b, hi, 0] if c["layout"] == "BNSD" else row[hi, b * -(-T // 128)]
                blocks = torch.zeros(0x10000, dtype=torch.bool, device="cuda")
                blocks[row.long()] = True
                ok = see & blocks[torch.arange(n, device="cuda") // c["BKV"]]
            q = s["q"][b, h] if c["layout"] == "BNSD" else s["q"][b * T:(b + 1) * T, h]
            x = (q.double() @ k[h // g].T) / math.sqrt(D)
            x = torch.where(ok, x, -math.inf)
            l = torch.logsumexp(x, -1)
            oo.append(torch.exp(x - torch.where(torch.isfinite(l), l, 0.0).unsqueeze(-1)) @ v[h // g])
            ll.append(l)
        outs.append(torch.stack(oo))
        lses.append(torch.stack(ll))
    o, l = torch.stack(outs), torch.stack(lses)  # [B, N1, T, ...]
    if c["layout"] != "BNSD":
        o, l = o.transpose(1, 2).flatten(0, 1), l.transpose(1, 2).flatten(0, 1)
    return o, l


def exact(case, seed):
    s = prepare(case, seed)
    return {"means": _exact_means, "select": _exact_select, "decode": _exact_decode}[case["op"]](s)
