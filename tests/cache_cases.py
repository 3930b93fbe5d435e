"""Small caches and plain 64-bit forms of the cache operators (block means,
block selection, few-token attention) for their tests."""
from __future__ import annotations

import math
from types import SimpleNamespace

import torch

import block_sparse_variable_b200 as bsa

NONE = 0xFFFF


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(layout="PA_BBND", N1=4, N2=2, D=128, qlens=(1,), kvlens=(100,), page=128, BKV=128, BQ=128,
         dtype=torch.bfloat16, seed=0, device="cuda", tail_rows=3, poison=True, interleaved=False):
    """A batch with its cache.  Rows that belong to no token (the rest of a
    page, rows past the used length, unused pages) hold NaN; the query tensor
    has `tail_rows` rows behind the last sequence (TND)."""
    g = torch.Generator().manual_seed(seed)
    B, fill = len(kvlens), float("nan") if poison else 0.0

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(dtype)

    s = SimpleNamespace(layout=layout, B=B, N1=N1, N2=N2, D=D, qlens=list(qlens), kvlens=list(kvlens), page=page,
                        BKV=BKV, BQ=BQ, dtype=dtype, device=device, g=g)
    s.kd = [normal(n, N2, D) for n in kvlens]
    s.vd = [normal(n, N2, D) for n in kvlens]
    s.qd = [normal(n, N1, D) for n in qlens]
    s.cu_q = s.cu_kv = s.used = s.table = None
    if layout == "PA_BBND":
        most = max(1, max(-(-n // page) for n in kvlens))
        total = sum(-(-n // page) for n in kvlens) + 2
        k = torch.full((total, page, N2, D), fill, dtype=dtype)
        v = torch.full((total, page, N2, D), fill, dtype=dtype)
        perm = torch.randperm(total, generator=g).tolist()
        table = torch.full((B, most + 1), -7, dtype=torch.int32)  # unused entries name no page
        for b, n in enumerate(kvlens):
            for x in range(-(-n // page)):
                pg = table[b, x] = perm.pop()
                m = min(page, n - x * page)
                k[pg, :m], v[pg, :m] = s.kd[b][x * page:x * page + m], s.vd[b][x * page:x * page + m]
        s.table = table.to(device)
        s.used = torch.tensor(kvlens, dtype=torch.int32, device=device)
    elif layout == "TND":
        k = torch.cat(s.kd + [torch.full((2, N2, D), fill, dtype=dtype)])
        v = torch.cat(s.vd + [torch.full((2, N2, D), fill, dtype=dtype)])
        s.cu_kv = cu(kvlens, device)
    else:
        S = max(kvlens) + 5
        k = torch.full((B, N2, S, D), fill, dtype=dtype)
        v = torch.full((B, N2, S, D), fill, dtype=dtype)
        for b, n in enumerate(kvlens):
            k[b, :, :n], v[b, :, :n] = s.kd[b].transpose(0, 1), s.vd[b].transpose(0, 1)
        s.used = torch.tensor(kvlens, dtype=torch.int32, device=device)
    if interleaved:  # k and v of a token side by side: row strides of 2 D
        kv = torch.stack((k, v), dim=-2).to(device)
        s.k, s.v = kv[..., 0, :], kv[..., 1, :]
    else:
        s.k, s.v = k.to(device), v.to(device)
    if layout == "BNSD":
        assert len(set(qlens)) == 1
        s.q = torch.stack([x.transpose(0, 1) for x in s.qd]).contiguous().to(device)
    else:
        s.q = torch.cat(s.qd + [torch.full((tail_rows, N1, D), fill, dtype=dtype)]).to(device)
        s.cu_q = cu(qlens, device)
    s.NB = max(1, max(-(-n // BKV) for n in kvlens))
    return s


def cu(lens, device):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64, device=device)


def params(s, **kw):
    kw = dict(block_shape=(s.BQ, s.BKV)) | kw
    return bsa.params_for("BNSD" if s.layout == "BNSD" else "TND", s.layout, s.N1, s.N2, **kw)


def where(s):
    return dict(cu_seqlens_kv=s.cu_kv, seqused_kv=s.used, block_table=s.table)


# ------------------------------------------------------------ plain 64-bit
def ref_means(s):
    """[B][N2, nk, D] means, and the mean of |k| beside each."""
    out = []
    for k in s.kd:
        parts = [k[j:j + s.BKV].double() for j in range(0, k.shape[0], s.BKV)]
        out.append((torch.stack([x.mean(0) for x in parts], 1), torch.stack([x.abs().mean(0) for x in parts], 1))
                   if parts else None)
    return out


def ref_select(s, means, W, rows, causal=False, sink=0, local=0):
    """Index rows [H, rows of the batch, W] as lists, by sorting."""
    g = s.N1 // s.N2
    H = s.N1 if rows == "query" else s.N2
    out = []
    for b in range(s.B):
        for i in range(-(-s.qlens[b] // s.BQ)):
            q = s.qd[b][i * s.BQ:(i + 1) * s.BQ].double().sum(0)  # [N1, D]
            if rows == "group":
                q = q.view(s.N2, g, s.D).sum(1)
            last = min(s.qlens[b], (i + 1) * s.BQ) - 1 + s.kvlens[b] - s.qlens[b]
            nk = -(-s.kvlens[b] // s.BKV)
            if causal:
                nk = 0 if last < 0 else min(nk, last // s.BKV + 1)
            row = []
            for h in range(H):
                m = means[b, h * s.N2 // H].cpu().double()
                def rank(j):
                    if j < sink or j >= nk - local:
                        return (0, 0.0, j)
                    x = float((m[j] * q[h]).sum())
                    return (2, 0.0, j) if math.isnan(x) else (1, -x, j)
                ids = sorted(sorted(range(nk), key=rank)[:W])
                row.append(ids + [NONE] * (W - len(ids)))
            out.append(row)
    return torch.tensor(out).transpose(0, 1) if out else None  # [H, R, W]


def accepted(row, nk):
    """The entries of an index row that take part."""
    out = []
    for e in row:
        if e != NONE and e < nk and (not out or e > out[-1]):
            out.append(e)
    return out


def ref_decode(s, index=None, tree=None, causal=False, scale=None, bad_pages=()):
    """Per batch: out, lse, sum P |v| / l and the error a score may have.
    index: [H][rows][W] lists; tree: [tokens of all sequences][words]."""
    scale = 1 / math.sqrt(s.D) if scale is None else scale
    g, at, row0, res = s.N1 // s.N2, 0, 0, []
    for b in range(s.B):
        n, T = s.kvlens[b], s.qlens[b]
        out = torch.zeros(T, s.N1, s.D, dtype=torch.float64)
        lse = torch.full((T, s.N1), -math.inf, dtype=torch.float64)
        mass, ds = torch.zeros(T, s.N1, s.D, dtype=torch.float64), torch.zeros(T, s.N1, dtype=torch.float64)
        u = torch.arange(n)
        node = u - (n - T)
        for t in range(T):
            ok = torch.ones(n, dtype=torch.bool)
            if causal:
                ok = node <= t
            if tree is not None:
                bits = [int(x) & (2 ** 64 - 1) for x in tree[at + t].tolist()]
                ok = torch.tensor([x < 0 or (x // 64 < len(bits) and bits[x // 64] >> (x % 64) & 1 == 1)
                                   for x in node.tolist()], dtype=torch.bool)
            for x in bad_pages:
                if x[0] == b:
                    ok = ok & (u // s.page != x[1])
            for h in range(s.N1):
                see = ok
                if index is not None:
                    H = len(index)
                    row = accepted(index[h * H // s.N1][row0 + t // s.BQ], -(-n // s.BKV))
                    keep = torch.zeros(max(1, -(-n // s.BKV)), dtype=torch.bool)
                    keep[row] = True
                    see = ok & keep[u // s.BKV]
                if n == 0 or not see.any():
                    continue
                k, v = s.kd[b][:, h // g].double()[see], s.vd[b][:, h // g].double()[see]
                q = s.qd[b][t, h].double()
                x = scale * (k @ q)
                lse[t, h] = torch.logsumexp(x, 0)
                p = torch.exp(x - lse[t, h])
                out[t, h], mass[t, h] = p @ v, p @ v.abs()
                ds[t, h] = float((k.abs() @ q.abs()).max()) * scale
        res.append((out, lse, mass, ds))
        at += T
        row0 += -(-T // s.BQ)
    return res


def check_decode(s, out, lse, ref):
    """Bounds by arithmetic: a weight is rounded once to the type (half a step
    of itself; for fp16 half the subnormal spacing, 2^-25, below 2^-14), out
    once more; a score is a sum of D fp32 products of which the largest error
    is (D + 4) 2^-24 of the sum of magnitudes, and the exponential's own is
    below 2^-21; sums over n keys add n 2^-24 of their magnitudes."""
    e, at = half_step(s.dtype), 0
    for b in range(s.B):
        T, n = s.qlens[b], s.kvlens[b]
        ro, rl, mass, ds = ref[b]
        o = (out[b].transpose(0, 1) if s.layout == "BNSD" else out[at:at + T]).double().cpu()
        l = (lse[b].transpose(0, 1) if s.layout == "BNSD" else lse[at:at + T]).double().cpu()
        at += T
        w = (s.D + 4) * 2.0 ** -24 * ds + 2.0 ** -21 + n * 2.0 ** -24  # relative error of a weight
        tiny = n * 2.0 ** -25 * (float(s.vd[b].abs().max()) if n else 0.0) if s.dtype == torch.float16 else 0.0
        tol = (e + 2 * w.unsqueeze(-1)) * mass * (1 + e) + e * ro.abs() + tiny + 1e-30
        assert torch.equal(torch.isneginf(l), torch.isneginf(rl))
        seen = ~torch.isneginf(rl)
        assert (o[~seen] == 0).all()
        assert torch.isfinite(o).all()
        assert ((o - ro).abs() <= tol).all(), float(((o - ro).abs() / tol).max())
        d = (l - rl).abs()[seen]
        assert (d <= (w[seen] * 2 + rl.abs()[seen] * 2.0 ** -22)).all(), float(d.max())


def random_tree(T, words, g, roots=0.1):
    """Ancestor bits; a few nodes are roots of their own."""
    rows, masks = [], []
    for j in range(T):
        up = 0 if j == 0 or float(torch.rand((), generator=g)) < roots else masks[int(torch.randint(0, j, (), generator=g))]
        masks.append(up | 1 << j)
        rows.append([m - (1 << 64) if m >> 63 else m for m in
                     ((masks[-1] >> (64 * w)) & (2 ** 64 - 1) for w in range(words))])
    return torch.tensor(rows, dtype=torch.int64).view(T, words)


def random_index(s, W, heads, messy=False):
    """[H][R][W]: random ascending blocks of every query block's sequence, the
    row's last slots unused; messy: unused slots anywhere, and entries that
    are out of range or not ascending."""
    out = [[] for _ in range(heads)]
    for b in range(s.B):
        nk = -(-s.kvlens[b] // s.BKV)
        for _ in range(-(-s.qlens[b] // s.BQ)):
            for h in range(heads):
                n = int(torch.randint(0, min(W, nk) + 1, (), generator=s.g))
                row = sorted(torch.randperm(nk, generator=s.g)[:n].tolist()) + [NONE] * (W - n)
                if messy:
                    row = [row[i] for i in torch.randperm(W, generator=s.g).tolist()]
                    row[int(torch.randint(0, W, (), generator=s.g))] = nk + 3
                out[h].append(row)
    return out


def index_tensor(s, rows):
    t = torch.tensor(rows, dtype=torch.int32, device=s.device)  # [H, R, W]
    if s.layout == "BNSD":
        t = t.view(t.shape[0], s.B, -1, t.shape[2]).transpose(0, 1)
    return t.contiguous().to(torch.uint16)
