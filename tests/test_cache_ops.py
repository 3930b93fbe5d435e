"""Block means, block selection and few-token attention over a cache, against
plain 64-bit forms, and their refusals (the latter without a GPU)."""
import math

import pytest
import torch

import block_sparse_variable_b200 as bsa
from tests import cache_cases as C

gpu = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# ----------------------------------------------------------------- refusals
def _code(fn):
    with pytest.raises(bsa.BsaError) as e:
        fn()
    return e.value.status


def test_workspace_sizes_and_empty_calls():
    s = C.make(qlens=(3, 1), kvlens=(300, 5), device="cpu", poison=False)
    P = C.params(s)
    means = torch.zeros(s.B, s.N2, s.NB, s.D, dtype=s.dtype)
    assert bsa.bsa_block_means_get_workspace(s.k, means, P, **C.where(s)) > 0
    index = torch.zeros(s.N2, 2, 4, dtype=torch.uint16)
    assert bsa.bsa_select_blocks_get_workspace(s.q, means, index, P, cu_seqlens_q=s.cu_q, seqused_kv=s.used) > 0
    assert bsa.bsa_decode_get_workspace(s.q, s.k, s.v, P, index=index, cu_seqlens_q=s.cu_q, seqused_kv=s.used,
                                        block_table=s.table) > 0


def test_refusals_means():
    s = C.make(kvlens=(300, 5), qlens=(1, 1), device="cpu", poison=False)
    P, w = C.params(s), C.where(s)
    m = torch.zeros(s.B, s.N2, s.NB, s.D, dtype=s.dtype)
    ask = bsa.bsa_block_means_get_workspace
    assert _code(lambda: ask(s.k, m.half(), P, **w)) == 161002
    assert _code(lambda: ask(s.k, m[:, :1], P, **w)) == 161002
    assert _code(lambda: ask(s.k, m[..., :64], P, **w)) == 161002
    assert _code(lambda: ask(s.k, m, P, seqused_kv=s.used)) == 161001             # no table
    assert _code(lambda: ask(s.k, m, P, block_table=s.table)) == 161001           # no lengths
    assert _code(lambda: ask(s.k, m, P, **w, first_kv=s.used[:1])) == 161002
    assert _code(lambda: ask(s.k, m, P, **w, first_kv=s.used.long())) == 161002
    assert _code(lambda: ask(s.k, m, C.params(s, block_shape=(128, 96)), **w)) == 161002
    assert _code(lambda: ask(s.k.to(torch.float8_e4m3fn), m, P, **w)) == 161003
    assert _code(lambda: ask(s.k[:, :64], m, P, **w)) == 161003                    # page of 64
    assert _code(lambda: ask(s.k[..., :32], m[..., :32], P, **w)) == 161003        # D = 32
    big = torch.empty(0, s.N2, 70000, s.D, dtype=s.dtype)
    assert _code(lambda: ask(s.k, big, P, seqused_kv=s.used[:0], block_table=s.table[:0])) == 161003


def test_refusals_select():
    s = C.make(kvlens=(300, 5), qlens=(3, 1), device="cpu", poison=False)
    P = C.params(s)
    m = torch.zeros(s.B, s.N2, s.NB, s.D, dtype=s.dtype)
    ix = torch.zeros(s.N2, 2, 4, dtype=torch.uint16)

    def ask(q=s.q, means=m, index=ix, params=P, **kw):
        a = dict(cu_seqlens_q=s.cu_q, seqused_kv=s.used) | kw
        return bsa.bsa_select_blocks_get_workspace(q, means, index, params, **a)
    assert ask() > 0
    assert _code(lambda: ask(cu_seqlens_q=None)) == 161001
    assert _code(lambda: ask(seqused_kv=None)) == 161001
    assert _code(lambda: ask(means=m[:1])) == 161002
    assert _code(lambda: ask(means=m.half())) == 161002
    assert _code(lambda: ask(index=ix[:1])) == 161002                              # heads neither N1 nor N2
    assert _code(lambda: ask(index=ix.view(torch.int16))) == 161002
    assert _code(lambda: ask(index=ix[0])) == 161002
    assert _code(lambda: ask(sink_blocks=-1)) == 161002
    assert _code(lambda: ask(local_blocks=-1)) == 161002
    assert _code(lambda: ask(q=s.q.float())) == 161002
    assert _code(lambda: ask(cu_seqlens_kv=s.cu_q)) == 161002                      # paged: no cu_seqlens_kv


def test_refusals_decode():
    s = C.make(kvlens=(300, 5), qlens=(3, 1), device="cpu", poison=False)
    P = C.params(s)
    tree = torch.zeros(s.q.shape[0], 1, dtype=torch.int64)
    ix = torch.zeros(s.N2, 2, 4, dtype=torch.uint16)

    def ask(q=s.q, k=s.k, v=s.v, params=P, **kw):
        a = dict(cu_seqlens_q=s.cu_q, seqused_kv=s.used, block_table=s.table) | kw
        return bsa.bsa_decode_get_workspace(q, k, v, params, **a)
    assert ask() > 0 and ask(index=ix) > 0 and ask(tree_mask=tree) > 0
    for missing in ("cu_seqlens_q", "seqused_kv", "block_table"):
        assert _code(lambda: ask(**{missing: None})) == 161001
    assert _code(lambda: ask(v=s.v.half())) == 161002
    assert _code(lambda: ask(v=s.v[:1])) == 161002
    assert _code(lambda: ask(q=s.q[:, :3])) == 161002
    assert _code(lambda: ask(q=s.q.to(torch.float8_e4m3fn))) == 161003
    assert _code(lambda: ask(tree_mask=tree, params=C.params(s, causal=True))) == 161002
    assert _code(lambda: ask(tree_mask=tree[:2])) == 161002
    assert _code(lambda: ask(tree_mask=tree.int())) == 161002
    assert _code(lambda: ask(index=ix[:, :, :0])) == 161002
    assert _code(lambda: ask(index=ix.int())) == 161002
    assert _code(lambda: ask(params=C.params(s, scale=-1.0))) == 161002
    assert _code(lambda: ask(params=C.params(s, scale=math.inf))) == 161002
    assert _code(lambda: ask(lse=torch.zeros(2, 4))) == 161002
    assert _code(lambda: ask(out=s.q[:3])) == 161002
    wide = torch.zeros(s.q.shape[0], s.N1, 132, dtype=s.dtype)[..., :128]          # row stride 132
    assert _code(lambda: ask(q=wide)) == 161002
    n = C.make("BNSD", kvlens=(200, 200), qlens=(70, 70), device="cpu", poison=False)
    shared = n.k[:1].expand(2, -1, -1, -1)                                         # one cache for two sequences
    assert _code(lambda: bsa.bsa_decode_get_workspace(n.q, shared, n.v, C.params(n), seqused_kv=n.used)) == 161003
    short = torch.zeros(2, 70, 1, dtype=torch.int64)                               # 64 bits for 70 nodes
    assert _code(lambda: bsa.bsa_decode_get_workspace(n.q, n.k, n.v, C.params(n), tree_mask=short,
                                                      seqused_kv=n.used)) == 161002


def test_host_tensors_are_refused_before_any_launch():
    s = C.make(kvlens=(300,), device="cpu", poison=False)
    with pytest.raises(ValueError):
        bsa.bsa_decode(s.q, s.k, s.v, C.params(s), cu_seqlens_q=s.cu_q, seqused_kv=s.used, block_table=s.table)
    with pytest.raises(ValueError):
        bsa.bsa_block_means(s.k, C.params(s), **C.where(s))


# -------------------------------------------------------------------- means
MEANS = [
    dict(kvlens=(1,), N2=1),
    dict(kvlens=(0, 127, 128, 129), page=128),
    dict(kvlens=(700, 3, 512), page=256, BKV=512, N2=3, N1=3, D=64, dtype=FP),
    dict(kvlens=(1025, 900), page=512, BKV=256, interleaved=True),
    dict(layout="TND", kvlens=(333, 0, 1, 2050), BKV=1024, D=64),
    dict(layout="TND", kvlens=(333, 50), dtype=FP, interleaved=True),
    dict(layout="BNSD", kvlens=(260, 0, 384), qlens=(1, 1, 1), N2=3, N1=6),
    dict(kvlens=(20000, 133, 0), N2=8),                                             # a warp a block
    dict(layout="TND", kvlens=(40007, 0, 1, 2050), N2=8, BKV=256, D=64, dtype=FP),
]


@gpu
@pytest.mark.parametrize("kw", MEANS, ids=str)
def test_means(kw):
    kw = dict(qlens=(1,) * len(kw["kvlens"])) | kw
    s = C.make(**kw, seed=3)
    ref = C.ref_means(s)
    mark = 7.0  # blocks that do not exist are left as they were
    means = torch.full((s.B, s.N2, s.NB + 1, s.D), mark, dtype=s.dtype, device="cuda")
    got, ws = bsa.bsa_block_means(s.k, C.params(s), **C.where(s), means=means)
    assert got.data_ptr() == means.data_ptr() and bsa.bsa_read_status(ws) == 0
    e = C.half_step(s.dtype)
    for b in range(s.B):
        nk = -(-s.kvlens[b] // s.BKV)
        assert (got[b, :, nk:] == mark).all()
        if nk:
            m, mag = ref[b]
            # fp32 sums of at most BKV values, one division, one rounding
            tol = e * m.abs() + (s.BKV + 2) * 2.0 ** -24 * mag * (1 + e) + 2.0 ** -25
            assert ((got[b, :, :nk].double().cpu() - m).abs() <= tol).all()


@gpu
@pytest.mark.parametrize("BKV", [128, 512])
def test_means_append_writes_the_new_tokens_blocks_only(BKV):
    s = C.make(kvlens=(1000, 128, 129, 5, 0), qlens=(1,) * 5, BKV=BKV, page=256)
    whole, _ = bsa.bsa_block_means(s.k, C.params(s), **C.where(s))
    first = torch.tensor([990, 127, 128, 0, 0], dtype=torch.int32, device="cuda")
    part = torch.full_like(whole, 9.0)
    bsa.bsa_block_means(s.k, C.params(s), **C.where(s), first_kv=first, means=part)
    for b, f in enumerate(first.tolist()):
        j, nk = f // BKV, -(-s.kvlens[b] // BKV)
        assert torch.equal(part[b, :, j:nk], whole[b, :, j:nk])
        assert (part[b, :, :j] == 9).all() and (part[b, :, nk:] == 9).all()


@gpu
def test_means_bad_values_are_flagged():
    s = C.make(kvlens=(400, 200), qlens=(1, 1), BKV=256)
    s.table[0, 1] = 999
    means, ws = bsa.bsa_block_means(s.k, C.params(s), **C.where(s))
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_PAGE
    m = s.kd[0][:128].double().mean(0)  # the block's other page
    assert ((means[0, :, 0].double().cpu() - m).abs() <= 2.0 ** -8 * m.abs() + 1e-4).all()
    s.used[0] = -1
    before = torch.full_like(means, 5.0)
    _, ws = bsa.bsa_block_means(s.k, C.params(s), **C.where(s), means=before)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN and (before[0] == 5).all()


# ---------------------------------------------------------------- selection
SELECT = [
    dict(qlens=(1, 1), kvlens=(2000, 131), W=5),
    dict(qlens=(1,), kvlens=(40000,), N1=8, N2=2, W=64, local=2, sink=1),
    dict(qlens=(300, 0, 129, 2), kvlens=(700, 100, 129, 1500), W=3, rows="query", dtype=FP),
    dict(qlens=(700, 513), kvlens=(700, 600), W=4, causal=True, BQ=256, D=64, N1=6),
    dict(qlens=(500,), kvlens=(300,), W=2, causal=True, local=1),  # leading rows see nothing
    dict(layout="TND", qlens=(260, 5), kvlens=(1300, 5), W=4, BKV=256, rows="query", causal=True, sink=2),
    dict(layout="BNSD", qlens=(300, 300), kvlens=(1100, 640), W=3, rows="query", N1=4, N2=4),
    dict(layout="BNSD", qlens=(2, 2), kvlens=(130000, 9), W=8, N1=2, N2=1, D=64, sink=3, local=3),
    dict(qlens=(1,), kvlens=(600,), W=1),
    dict(qlens=(1, 3), kvlens=(0, 600), W=2, sink=1),
    dict(qlens=(900, 0, 129, 2, 0), kvlens=(1700, 100, 129, 1500, 9), W=3, rows="query", dtype=FP),
    dict(layout="TND", qlens=(900, 5), kvlens=(1300, 5), W=4, BKV=256, rows="query", causal=True, sink=2),
    dict(qlens=(256, 131), kvlens=(1300, 5000), W=4, N1=16, N2=2),                  # 1024 query rows a row
    dict(qlens=(400,) + (1,) * 9, kvlens=(3000,) + (700,) * 9, W=3, causal=True),   # a prompt among single tokens
]


def _select(s, means, kw, **over):
    H = s.N1 if kw.get("rows", "group") == "query" else s.N2
    rows = sum(-(-n // s.BQ) for n in s.qlens)
    a = dict(width=kw["W"], index_heads=H, rows=rows, sink_blocks=kw.get("sink", 0),
             local_blocks=kw.get("local", 0), cu_seqlens_q=s.cu_q, cu_seqlens_kv=s.cu_kv, seqused_kv=s.used) | over
    return bsa.bsa_select_blocks(s.q, means, C.params(s, causal=kw.get("causal", False)), **a)


def _as_rows(s, index):
    t = index.to(torch.int32).cpu() & 0xFFFF
    if s.layout == "BNSD":
        t = t.transpose(0, 1).reshape(t.shape[1], -1, t.shape[-1])
    return t


def _split(kw):
    return {k: v for k, v in kw.items() if k not in ("W", "rows", "causal", "sink", "local")}


@gpu
@pytest.mark.parametrize("kw", SELECT, ids=str)
def test_select(kw):
    s = C.make(**_split(kw), seed=5)
    means = torch.randn(s.B, s.N2, s.NB, s.D, generator=s.g).to(s.dtype).cuda()
    for b, n in enumerate(s.kvlens):
        means[b, :, -(-n // s.BKV):] = float("nan")  # no candidates
    index, ws = _select(s, means, kw)
    ref = C.ref_select(s, means, kw["W"], kw.get("rows", "group"), kw.get("causal", False), kw.get("sink", 0),
                       kw.get("local", 0))
    assert bsa.bsa_read_status(ws) == 0
    assert torch.equal(_as_rows(s, index), ref.int())


@gpu
@pytest.mark.parametrize("W", [1, 3, 40])
@pytest.mark.parametrize("kvlen", [9000, 50000, 140000])
def test_select_ties_infinities_and_nan(W, kvlen):
    """Scores of whole numbers are exact, so equal ones are ties."""
    s = C.make(qlens=(1, 130), kvlens=(kvlen, 5000), N1=4, N2=2, D=64, seed=8, poison=False)
    for x in s.qd:
        x.copy_(x.sign())
    s.q = torch.cat(s.qd).cuda()
    means = torch.randint(-1, 2, (s.B, s.N2, s.NB, s.D), generator=s.g).to(s.dtype)
    means[0, 0, 3] = float("nan")
    means[0, 0, 5, 0] = float("inf")
    means[0, 1, 6, 1] = -float("inf")
    means[0, :, 20:30] = 0.0
    means[1, 1] = -0.0
    means = means.cuda()
    kw = dict(W=W)
    index, _ = _select(s, means, kw)
    assert torch.equal(_as_rows(s, index), C.ref_select(s, means, W, "group").int())


@gpu
@pytest.mark.parametrize("T", [1, 200])
def test_select_close_scores_are_ordered(T):
    """Two blocks whose scores differ by 1 part in 10^9."""
    s = C.make(qlens=(T,), kvlens=(512,), N1=1, N2=1, D=64, dtype=FP, poison=False, tail_rows=0)
    s.q[:] = 1.0
    s.q[:, 0, 1] = 2.0 ** -10
    m = torch.zeros(1, 1, 4, 64, dtype=FP, device="cuda")
    m[0, 0, :, 0] = 1024.0
    m[0, 0, 2, 1] = 2.0 ** -12
    index, _ = _select(s, m, dict(W=1))
    assert (index.to(torch.int32) == 2).all()


@gpu
@pytest.mark.parametrize("T", [1, 150])
@pytest.mark.parametrize("dtype, scale", [(BF, 1e37), (BF, 1e-37), (FP, 6e4), (FP, 1e-7)])
def test_select_at_the_ends_of_the_range(T, dtype, scale):
    """Products that pass 32-bit floats, and values below the normal ones."""
    s = C.make(qlens=(T, T), kvlens=(5000, 2600), N1=4, N2=2, D=64, dtype=dtype, seed=13, poison=False, tail_rows=0)
    s.qd = [(x.double() * scale).clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype) for x in s.qd]
    s.q = torch.cat(s.qd).cuda()
    means = (torch.randn(s.B, s.N2, s.NB, s.D, generator=s.g).double() * scale / 8).to(dtype).cuda()
    index, _ = _select(s, means, dict(W=7))
    assert torch.equal(_as_rows(s, index), C.ref_select(s, means, 7, "group").int())


@gpu
def test_select_bad_lengths_and_missing_rows():
    s = C.make(qlens=(300, 200), kvlens=(700, 700), seed=2)
    means = torch.randn(2, 2, s.NB, s.D, generator=s.g).to(s.dtype).cuda()
    full, ws = _select(s, means, dict(W=2))
    index, ws = _select(s, means, dict(W=2), rows=4)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX
    assert torch.equal(index.view(torch.int16), full[:, :4].view(torch.int16))
    s.used[0] = 128 * s.NB + 1
    _, ws = _select(s, means, dict(W=2))
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN
    extra = torch.full((2, 9, 2), 77, dtype=torch.int16, device="cuda").view(torch.uint16)
    s.used[0] = 700
    _select(s, means, dict(W=2), index=extra)
    assert (extra[:, 5:].view(torch.int16) == 77).all()
    assert torch.equal(extra[:, :5].view(torch.int16), full.view(torch.int16))


# ------------------------------------------------------------------- decode
DECODE = [
    dict(kvlens=(1,)),
    dict(kvlens=(0, 1, 64, 65, 127, 128, 129), qlens=(1,) * 7),
    dict(kvlens=(1000,), N1=32, N2=8, dtype=FP),
    dict(kvlens=(4000, 33, 700), qlens=(1, 1, 1), N1=6, N2=2, D=64, page=256),
    dict(kvlens=(300, 2000, 10), qlens=(2, 0, 5), N1=8, N2=2),                     # ragged queries
    dict(kvlens=(777, 40), qlens=(33, 7), N1=12, N2=4, mask="causal", D=64, dtype=FP),
    dict(kvlens=(3, 200), qlens=(8, 8), mask="causal"),                             # more drafts than keys
    dict(kvlens=(500, 90), qlens=(24, 24), mask="tree", N1=8, N2=2),
    dict(kvlens=(300, 1200), qlens=(100, 70), mask="tree", N1=6, N2=2, dtype=FP, page=512),
    dict(kvlens=(700, 300), qlens=(100, 33), mask="tree", words=1, N1=2, N2=1),     # nodes past the words
    dict(layout="BNSD", kvlens=(130, 700), qlens=(3, 3), N1=4, N2=4, interleaved=True),
    dict(layout="BNSD", kvlens=(1500, 40), qlens=(24, 24), N1=16, N2=4, D=64, mask="tree"),
    dict(layout="TND", kvlens=(130, 0, 700), qlens=(2, 3, 1), N1=3, N2=1, interleaved=True),
    dict(layout="TND", kvlens=(600, 90), qlens=(200, 90), N1=4, N2=2, mask="causal"),
    dict(kvlens=(900, 300), qlens=(40, 1), N1=64, N2=8, mask="causal"),              # wide groups
    # selected blocks
    dict(kvlens=(3000, 400), qlens=(1, 1), W=4),
    dict(kvlens=(3000, 400, 0), qlens=(1, 3, 2), W=7, heads="query", N1=6, N2=2, dtype=FP),
    dict(kvlens=(9000, 4100), qlens=(2, 1), W=5, BKV=512, page=256, D=64),
    dict(kvlens=(9000, 700), qlens=(1, 1), W=40, messy=True),
    dict(kvlens=(2000, 700), qlens=(300, 10), W=6, N1=4, N2=2, messy=True, mask="causal"),
    dict(kvlens=(2000, 700), qlens=(20, 130), W=6, N1=6, N2=2, mask="tree", heads="query"),
    dict(layout="BNSD", kvlens=(2000, 700), qlens=(5, 5), W=6, mask="tree", N1=8, N2=1, BKV=256),
    dict(layout="TND", kvlens=(2000, 700), qlens=(5, 150), W=3, N1=16, N2=1, BKV=1024, interleaved=True),
]


def _decode_inputs(kw):
    extra = ("W", "heads", "mask", "messy", "words")
    s = C.make(**(dict(qlens=(1,) * len(kw["kvlens"])) | {k: v for k, v in kw.items() if k not in extra}), seed=11)
    rows = tree = None
    if "W" in kw:
        rows = C.random_index(s, kw["W"], s.N1 if kw.get("heads") == "query" else s.N2, kw.get("messy", False))
    if kw.get("mask") == "tree":
        words = kw.get("words", -(-max(s.qlens) // 64))
        tree = torch.cat([C.random_tree(T, words, s.g) for T in s.qlens])
        tree[0] = 0  # a node that sees no draft, not even itself
    return s, rows, tree


def _decode(s, rows, tree, causal, **over):
    dev_tree = None
    if tree is not None:
        dev_tree = tree.view(s.B, -1, tree.shape[1]) if s.layout == "BNSD" else \
            torch.cat([tree, torch.zeros(s.q.shape[0] - tree.shape[0], tree.shape[1], dtype=torch.int64)])
        dev_tree = dev_tree.cuda()
    a = dict(index=None if rows is None else C.index_tensor(s, rows), tree_mask=dev_tree, cu_seqlens_q=s.cu_q,
             **C.where(s)) | over
    return bsa.bsa_decode(s.q, s.k, s.v, C.params(s, causal=causal), **a)


@gpu
@pytest.mark.parametrize("kw", DECODE, ids=str)
def test_decode(kw):
    s, rows, tree = _decode_inputs(kw)
    causal = kw.get("mask") == "causal"
    out = torch.full_like(s.q, 3.0)
    out, lse, ws = _decode(s, rows, tree, causal, out=out)
    assert bsa.bsa_read_status(ws) in ((0, bsa.FLAG_BAD_INDEX) if kw.get("messy") else (0,))
    C.check_decode(s, out, lse, C.ref_decode(s, rows, tree, causal))
    if s.layout != "BNSD":
        assert (out[sum(s.qlens):] == 3).all()  # rows behind the last sequence
    again, lse2, _ = _decode(s, rows, tree, causal, workspace=ws)
    n = sum(s.qlens) if s.layout != "BNSD" else None
    assert torch.equal(again[:n], out[:n]) and torch.equal(lse2[:n], lse[:n])


@gpu
def test_decode_flags():
    s = C.make(kvlens=(1000, 300), qlens=(1, 1))
    s.table[0, 3] = 1 << 20
    out, lse, ws = _decode(s, None, None, False)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_PAGE
    C.check_decode(s, out, lse, C.ref_decode(s, bad_pages=[(0, 3)]))
    # a page that no row selects raises nothing; an entry that is out of range does
    rows = [[[0, 1], [0, 2]]] * s.N2
    _, _, ws = _decode(s, rows, None, False)
    assert bsa.bsa_read_status(ws) == 0
    rows = [[[0, 1], [0, 5]]] * s.N2
    _, _, ws = _decode(s, rows, None, False)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX
    # too few index rows: the second sequence selects nothing
    out, lse, ws = _decode(s, [[[0, 1]]] * s.N2, None, False)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all() and torch.isfinite(lse[0]).all()
    s.used[0] = s.table.shape[1] * s.page + 1
    out, lse, ws = _decode(s, None, None, False)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.isfinite(lse[1]).all()


@gpu
def test_decode_scale_no_lse_and_own_buffers():
    s = C.make(kvlens=(700,), qlens=(4,), N1=8, N2=2)
    P = C.params(s, scale=0.3, return_lse=False)
    store = torch.zeros(s.q.shape[0], s.N1, 2 * s.D, dtype=s.dtype, device="cuda")
    out, lse, _ = bsa.bsa_decode(s.q, s.k, s.v, P, cu_seqlens_q=s.cu_q, **C.where(s), out=store[..., s.D:])
    assert lse is None and (store[..., :s.D] == 0).all()
    _, lse, _ = bsa.bsa_decode(s.q, s.k, s.v, C.params(s, scale=0.3), cu_seqlens_q=s.cu_q, **C.where(s))
    C.check_decode(s, out, lse, C.ref_decode(s, scale=0.3))


@gpu
def test_decode_many_short_sequences():
    """More units than blocks of the grid: most finish inside one block."""
    g = torch.Generator().manual_seed(0)
    kvlens = torch.randint(0, 90, (700,), generator=g).tolist()
    s = C.make(kvlens=kvlens, qlens=(1,) * 700, N1=2, N2=2, D=64)
    out, lse, ws = _decode(s, None, None, False)
    assert bsa.bsa_read_status(ws) == 0
    C.check_decode(s, out, lse, C.ref_decode(s))


@gpu
def test_decode_long_cache_past_32_bit_offsets():
    """A cache of more than 2^31 elements; the pages in use sit at its end."""
    D, N2, page = 128, 8, 1024
    pages = 2 ** 31 // (page * N2 * D) + 40
    k = torch.empty(pages, page, N2, D, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    s = C.make(kvlens=(5000,), qlens=(1,), N1=16, N2=N2, page=page, seed=4)
    n = s.k.shape[0]
    k[-n:], v[-n:] = s.k, s.v
    s.k, s.v = k, v
    s.table[:, :5] += pages - n
    out, lse, ws = _decode(s, None, None, False)
    assert bsa.bsa_read_status(ws) == 0
    C.check_decode(s, out, lse, C.ref_decode(s))
    means, _ = bsa.bsa_block_means(k, C.params(s), **C.where(s))
    m, mag = C.ref_means(s)[0]
    assert ((means[0, :, :m.shape[1]].double().cpu() - m).abs() <= 2.0 ** -8 * m.abs() + 2.0 ** -16 * mag).all()


# ------------------------------------------------------------ used together
@gpu
def test_generation_step_by_step():
    """A prompt, then tokens one at a time: means are appended to, blocks are
    chosen from them and attended over."""
    s = C.make(kvlens=(900, 260), qlens=(1, 1), N1=8, N2=2, seed=21)
    P = C.params(s)
    used = s.used - 3
    means, ws_m = bsa.bsa_block_means(s.k, P, block_table=s.table, seqused_kv=used)
    index = ws_s = ws_d = None
    for step in range(1, 4):
        first, used = used, used + 1
        means, ws_m = bsa.bsa_block_means(s.k, P, block_table=s.table, seqused_kv=used, first_kv=first, means=means,
                                          workspace=ws_m)
        index, ws_s = bsa.bsa_select_blocks(s.q, means, P, width=3, rows=2, sink_blocks=1, local_blocks=1,
                                            cu_seqlens_q=s.cu_q, seqused_kv=used, workspace=ws_s)
        out, lse, ws_d = bsa.bsa_decode(s.q, s.k, s.v, P, index=index, cu_seqlens_q=s.cu_q, seqused_kv=used,
                                        block_table=s.table, workspace=ws_d)
        fresh, _ = bsa.bsa_block_means(s.k, P, block_table=s.table, seqused_kv=used)
        nk = [-(-n // s.BKV) for n in used.tolist()]
        for b in range(2):
            assert torch.equal(means[b, :, :nk[b]], fresh[b, :, :nk[b]])
        t = C.make(kvlens=(900, 260), qlens=(1, 1), N1=8, N2=2, seed=21)
        t.kvlens = used.tolist()
        t.kd, t.vd = [k[:n] for k, n in zip(t.kd, t.kvlens)], [v[:n] for v, n in zip(t.vd, t.kvlens)]
        rows = C.ref_select(t, means, 3, "group", sink=1, local=1)
        assert torch.equal(_as_rows(s, index), rows.int())
        C.check_decode(t, out, lse, C.ref_decode(t, rows.tolist()))


@gpu
def test_selected_blocks_in_training():
    """The index of the selection through bsa_fwd and bsa_bwd: outputs and
    gradients against 64-bit autograd over the same blocks."""
    s = C.make("TND", qlens=(300, 130), kvlens=(300, 130), N1=4, N2=2, D=64, tail_rows=0, poison=False)
    P = C.params(s, causal=True)
    means, _ = bsa.bsa_block_means(s.k, P, cu_seqlens_kv=s.cu_kv)
    index, _ = bsa.bsa_select_blocks(s.q, means, P, width=2, rows=5, local_blocks=1, cu_seqlens_q=s.cu_q,
                                     cu_seqlens_kv=s.cu_kv)
    k, v = s.k[:430].contiguous(), s.v[:430].contiguous()
    out, lse, _ = bsa.bsa_fwd(s.q, k, v, index, P, cu_seqlens_q=s.cu_q, cu_seqlens_kv=s.cu_kv)
    dout = torch.randn(s.q.shape, generator=s.g).to(s.dtype).cuda()
    dq, dk, dv, _ = bsa.bsa_bwd(s.q, k, v, out, dout, lse, index, P, cu_seqlens_q=s.cu_q, cu_seqlens_kv=s.cu_kv)
    # the same rows through the few-token attention
    out2, lse2, _ = bsa.bsa_decode(s.q, k, v, P, index=index, cu_seqlens_q=s.cu_q, cu_seqlens_kv=s.cu_kv)
    rows = (index.to(torch.int32).cpu() & 0xFFFF).tolist()
    C.check_decode(s, out2, lse2, C.ref_decode(s, rows, causal=True))
    at = 0
    for b, n in enumerate(s.qlens):
        q, kk, vv = (x.double().requires_grad_() for x in (s.qd[b], s.kd[b], s.vd[b]))
        x = torch.einsum("thd,uhd->htu", q, kk.repeat_interleave(2, 1)) / 8.0
        ok = torch.zeros(4, n, n, dtype=torch.bool)
        for h in range(4):
            for t in range(n):
                keep = C.accepted(rows[h // 2][(0, 3)[b] + t // 128], 3)
                ok[h, t] = torch.tensor([u <= t and u // 128 in keep for u in range(n)])
        x = x.masked_fill(~ok, -math.inf)
        o = torch.einsum("htu,uhd->thd", torch.softmax(x, -1), vv.repeat_interleave(2, 1))
        o.backward(dout[at:at + n].double().cpu())
        for got, want in ((dq, q.grad), (dk, kk.grad), (dv, vv.grad)):
            d = got[at:at + n].double().cpu() - want
            assert (d.abs() <= 2e-2 * want.abs().clamp(min=1)).all()
        at += n


@gpu
def test_other_stream_and_captured_replay():
    s, rows, tree = _decode_inputs(dict(kvlens=(2000, 700), qlens=(5, 5), N1=8, N2=2, W=6, mask="tree"))
    t, _, _ = _decode_inputs(dict(kvlens=(2000, 700), qlens=(5, 5), N1=8, N2=2))
    plain, plain_lse, ws = _decode(s, rows, tree, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b, _ = _decode(s, rows, tree, False)
    side.synchronize()
    assert torch.equal(a[:10], plain[:10]) and torch.equal(b[:10], plain_lse[:10])
    means = torch.randn(2, 2, s.NB, s.D, generator=s.g).to(s.dtype).cuda()
    P = C.params(s)
    out, lse = torch.zeros_like(s.q), torch.zeros(s.q.shape[:2], device="cuda")
    index = torch.zeros(s.N2, 2, 6, dtype=torch.int16, device="cuda").view(torch.uint16)
    w_s = torch.empty(bsa.bsa_select_blocks_get_workspace(s.q, means, index, P, cu_seqlens_q=s.cu_q,
                                                          seqused_kv=s.used), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsa.bsa_select_blocks(s.q, means, P, cu_seqlens_q=s.cu_q, seqused_kv=s.used, index=index, workspace=w_s)
        bsa.bsa_decode(s.q, s.k, s.v, P, index=index, cu_seqlens_q=s.cu_q, **C.where(s), out=out, lse=lse,
                       workspace=ws)
    for lens in ([2000, 700], [130, 700], [1999, 1]):  # lengths change between replays
        s.used.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ix, _ = bsa.bsa_select_blocks(s.q, means, P, width=6, rows=2, cu_seqlens_q=s.cu_q, seqused_kv=s.used)
        o, l, _ = bsa.bsa_decode(s.q, s.k, s.v, P, index=ix, cu_seqlens_q=s.cu_q, **C.where(s))
        assert torch.equal(ix.view(torch.int16), index.view(torch.int16))
        assert torch.equal(o[:10], out[:10]) and torch.equal(l[:10], lse[:10])


@gpu
def test_made_tensors_are_made_on_the_given_stream():
    s = C.make(kvlens=(1500, 700), qlens=(300, 1), seed=21)
    P = C.params(s)
    m0 = bsa.bsa_block_means(s.k, P, **C.where(s))[0]
    kw = dict(cu_seqlens_q=s.cu_q, seqused_kv=s.used)
    i0 = bsa.bsa_select_blocks(s.q, m0, P, width=3, **kw)[0]
    o0 = bsa.bsa_decode(s.q, s.k, s.v, P, index=i0, block_table=s.table, **kw)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)  # the current stream is busy: a fill on it comes after the kernels
        m = bsa.bsa_block_means(s.k, P, **C.where(s), stream=given)[0]
        i = bsa.bsa_select_blocks(s.q, m, P, width=3, **kw, stream=given)[0]
        o = bsa.bsa_decode(s.q, s.k, s.v, P, index=i, block_table=s.table, **kw, stream=given)[0]
        torch.cuda.synchronize()
        n = sum(s.qlens)  # rows of no sequence are not written
        assert torch.equal(m, m0) and torch.equal(i.view(torch.int16), i0.view(torch.int16))
        assert torch.equal(o[:n], o0[:n])


@gpu
def test_empty_calls_report_a_clear_status():
    s = C.make(kvlens=(300, 5), qlens=(3, 1), poison=False)
    P, dev = C.params(s), "cuda"

    def dirty():
        return torch.full((1 << 20,), 255, dtype=torch.uint8, device=dev)
    none = torch.zeros(1, dtype=torch.int64, device=dev)
    used = torch.zeros(0, dtype=torch.int32, device=dev)
    # no sequences
    m = torch.zeros(0, s.N2, 3, s.D, dtype=s.dtype, device=dev)
    ws = bsa.bsa_block_means(s.k, P, seqused_kv=used, block_table=s.table[:0], means=m, workspace=dirty())[1]
    assert bsa.bsa_read_status(ws) == 0
    ws = bsa.bsa_select_blocks(s.q[:0], m, P, width=2, cu_seqlens_q=none, seqused_kv=used, workspace=dirty())[1]
    assert bsa.bsa_read_status(ws) == 0
    ws = bsa.bsa_decode(s.q[:0], s.k, s.v, P, cu_seqlens_q=none, seqused_kv=used, block_table=s.table[:0],
                        workspace=dirty())[2]
    assert bsa.bsa_read_status(ws) == 0
    # sequences without query tokens
    zero = torch.zeros(s.B + 1, dtype=torch.int64, device=dev)
    ws = bsa.bsa_decode(s.q[:0], s.k, s.v, P, cu_seqlens_q=zero, seqused_kv=s.used, block_table=s.table,
                        workspace=dirty())[2]
    assert bsa.bsa_read_status(ws) == 0
    # no room for the blocks, no rows for the query blocks
    m = torch.zeros(s.B, s.N2, 0, s.D, dtype=s.dtype, device=dev)
    ws = bsa.bsa_block_means(s.k, P, **C.where(s), means=m, workspace=dirty())[1]
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN
    m = torch.zeros(s.B, s.N2, s.NB, s.D, dtype=s.dtype, device=dev)
    ws = bsa.bsa_select_blocks(s.q, m, P, width=2, rows=0, cu_seqlens_q=s.cu_q, seqused_kv=s.used,
                               workspace=dirty())[1]
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX


@gpu
def test_two_captured_graphs_share_a_workspace():
    # other lengths, masks and kernels behind the same buffer, replayed in turn
    a = C.make(kvlens=(3000, 40), qlens=(1, 1), N1=8, N2=2, seed=31)
    b = C.make(kvlens=(900, 2600), qlens=(40, 17), N1=8, N2=2, seed=32)
    calls, want = [], []
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    for s, causal in ((a, False), (b, True)):
        def call(s=s, causal=causal, out=torch.empty_like(s.q), lse=torch.empty(s.q.shape[:2], device="cuda")):
            return bsa.bsa_decode(s.q, s.k, s.v, C.params(s, causal=causal), cu_seqlens_q=s.cu_q,
                                  seqused_kv=s.used, block_table=s.table, out=out, lse=lse, workspace=ws)[:2]
        calls.append(call)
        want.append([x.clone() for x in call()])
    graphs, got = [], []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1, 0)):
        for x in got:
            x[0].zero_(), x[1].zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert bsa.bsa_read_status(ws) == 0
        for i in (0, 1):
            valid = slice(0, int((a, b)[i].cu_q[-1]))
            assert torch.equal(got[i][0][valid], want[i][0][valid]) and torch.equal(got[i][1][valid], want[i][1][valid])
