"""The cache operators at the ends of what they accept: lengths that contradict
the storage, sizes near the limits, rules that switch kernels."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest
import torch

import block_sparse_variable_b200 as bsa
from tests import cache_cases as C
from tests.test_cache_ops import _as_rows, _decode, _select

gpu = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def test_line_arithmetic(tmp_path):
    """Division of a line of work, on the host (tests/line_check.cpp)."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    pkg = os.path.dirname(bsa.LIB_PATH)
    exe = str(tmp_path / "line_check")
    subprocess.check_call([cxx, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(pkg, "csrc"),
                           os.path.join(os.path.dirname(__file__), "line_check.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok"


def test_package_works_without_the_native_part_of_the_binding(tmp_path):
    """A package without _binding.so imports; the passes and the workspace
    queries work, a call of a cache operator says what is missing."""
    pkg = os.path.dirname(bsa.LIB_PATH)
    copy = tmp_path / "block_sparse_variable_b200"
    copy.mkdir()
    shutil.copy(os.path.join(pkg, "__init__.py"), copy)
    os.symlink(bsa.LIB_PATH, copy / "libbsa.so")
    code = """
import torch, block_sparse_variable_b200 as bsa
q = torch.zeros(1, 2, 200, 64, dtype=torch.bfloat16)
ix = torch.zeros(1, 2, 2, 2, dtype=torch.uint16)
P = bsa.params_for("BNSD", "BNSD", 2)
assert bsa.bsa_fwd_get_workspace(q, q, q, ix, P) > 0
assert bsa.bsa_decode_get_workspace(q, q, q, P) > 0
try:
    bsa.bsa_decode(q, q, q, P)
except ImportError as e:
    assert "_binding.so" in str(e) and "build.py" in str(e), e
    print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok"


def test_native_part_is_rebuilt_for_another_torch(monkeypatch, tmp_path):
    import importlib.util
    spec = importlib.util.spec_from_file_location("bsa_build", os.path.join(os.path.dirname(bsa.LIB_PATH), "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    key = tmp_path / "binding.txt"
    monkeypatch.setattr(b, "BINDING_KEY", str(key))
    monkeypatch.setattr(b, "_stale_file", lambda out, inputs: False)  # the sources are as they were
    assert b.binding_stale()
    key.write_text(b._binding_key())
    assert not b.binding_stale()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert b.binding_stale()


def test_tensor_memory_is_taken_after_the_wait():
    """A block that waits for the kernel before it must hold no tensor memory:
    that kernel's blocks, which may be on the same SM, take theirs while they run."""
    csrc = os.path.join(os.path.dirname(bsa.LIB_PATH), "csrc")
    seen = 0
    for name in sorted(os.listdir(csrc)):
        if not name.endswith(".cu"):
            continue
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for kernel in text.split("__global__")[1:]:
            if "tmem_alloc(" in kernel:
                seen += 1
                assert 0 <= kernel.find("griddep_wait();") < kernel.find("tmem_alloc("), name
    assert seen >= 4


def _decode_shapes(T, B, N1, N2, pages, BKV, W):
    """Status of bsa_decode_get_workspace for a paged call of these sizes (no memory behind it)."""
    d = {"q": ((T, N1, 64), BF), "k": ((1, 128, N2, 64), BF), "v": ((1, 128, N2, 64), BF),
         "index": None if W is None else ((N2, B, W), torch.uint16), "tree": None, "cu_q": ((B + 1,), torch.int64),
         "cu_kv": None, "used": ((B,), torch.int32), "table": ((B, pages), torch.int32), "out": ((T, N1, 64), BF),
         "lse": ((T, N1), torch.float32)}
    d = [None if x is None else bsa.describe_shape(*x) for x in d.values()]
    refs = [None if x is None else ctypes.byref(x) for x in d]
    prm, n = bsa.params_for("TND", "PA_BBND", N1, N2, (128, BKV)).c(), ctypes.c_size_t(0)
    return bsa.lib().bsa_decode_get_workspace(*refs[:9], ctypes.byref(prm), *refs[9:], ctypes.byref(n))


def test_decode_refuses_more_chunks_than_the_line_counts():
    """280 million single tokens before up to 128 tokens: 2 chunks a sequence of
    the whole cache or of one selected block of 128 tokens, 16 of a block of 1024."""
    n = 280_000_000
    assert _decode_shapes(n, n, 1, 1, 1, 1024, None) == 0
    assert _decode_shapes(n, n, 1, 1, 1, 128, 1) == 0
    assert _decode_shapes(n, n, 1, 1, 1, 1024, 1) == 161003


def test_misaligned_lengths_tables_and_indices_are_refused():
    """A load from an address that is no multiple of its size faults the GPU."""
    s = C.make(kvlens=(300, 5), qlens=(3, 1), device="cpu", poison=False)
    P, lib = C.params(s), bsa.lib()
    means = torch.zeros(s.B, s.N2, s.NB, s.D, dtype=s.dtype)
    ix = torch.zeros(s.N2, 2, 4, dtype=torch.uint16)
    tree = torch.zeros(s.q.shape[0], 1, dtype=torch.int64)
    lse = torch.zeros(s.q.shape[:2])
    calls = (  # entry, tensors, place of the params, scalars after it, tensors of whole numbers or 32-bit floats
        ("bsa_block_means", (s.k, None, s.used, s.table, s.used, means), 5, (), (2, 3, 4)),
        ("bsa_select_blocks", (s.q, means, s.cu_q, None, s.used, ix), 5, (0, 0), (2, 4, 5)),
        ("bsa_decode", (s.q, s.k, s.v, ix, tree, s.cu_q, None, s.used, s.table, s.q, lse), 9, (), (3, 4, 5, 7, 8, 10)),
        ("bsa_fwd", (s.q, s.k, s.v, ix, s.cu_q, None, s.used, s.table, s.q, lse), 8, (), (3, 4, 6, 7, 9)),
    )
    for name, tensors, at, extra, whole in calls:
        def ask(off=None):
            d = [bsa.describe(t) for t in tensors]
            if off is not None:
                d[off].data += 1
            refs = [None if x is None else ctypes.byref(x) for x in d]
            n, prm = ctypes.c_size_t(0), P.c()
            return getattr(lib, name + "_get_workspace")(*refs[:at], ctypes.byref(prm), *extra, *refs[at:], ctypes.byref(n))
        assert ask() == 0, name
        for i in whole:
            assert ask(i) == 161002, (name, i)


# ------------------------------------------------- sequences that overlap
@gpu
@pytest.mark.parametrize("N1", [2, 32])  # tiles of 16 and of 128 rows
@pytest.mark.parametrize("W", [None, 3])
def test_decode_overlapping_sequences(N1, W):
    """cu_seqlens that decrease: a pair that does counts as length 0, rows of
    one sequence alone are right."""
    s = C.make(kvlens=(500, 300, 900), qlens=(6, 0, 7), N1=N1, N2=2, tail_rows=0, seed=17)
    s.qd[2][:2] = s.qd[0][4:]
    s.q = torch.cat([s.qd[0], s.qd[2][2:]]).cuda()
    s.cu_q = torch.tensor([0, 6, 4, 11], device="cuda")  # rows 4 and 5 belong to two sequences
    rows = None if W is None else C.random_index(s, W, s.N2)
    out, lse, ws = _decode(s, rows, None, False)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN
    ref = C.ref_decode(s, rows)
    first, last = ref[0], ref[2]
    t = C.make(kvlens=(500, 900), qlens=(4, 5), N1=N1, N2=2, tail_rows=0)
    t.kd, t.vd = [s.kd[0], s.kd[2]], [s.vd[0], s.vd[2]]
    C.check_decode(t, torch.cat([out[:4], out[6:]]), torch.cat([lse[:4], lse[6:]]),
                   [[x[:4] for x in first], [x[2:] for x in last]])


@gpu
@pytest.mark.parametrize("N1, pages", [(64, 2048), (256, 8192)])  # tiles of 16 and of 128 rows
def test_decode_overlapping_sequences_past_the_line(N1, pages):
    """Every other sequence has all query tokens: more chunks than 32 bits count
    (an empty line, nothing written)."""
    T, B, N2, D = 1000, 999, 8, 64
    q = torch.zeros(T, N1, D, dtype=BF, device="cuda")
    k = torch.zeros(1, 128, N2, D, dtype=BF, device="cuda")
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda").expand(B, pages)
    used = torch.full((B,), pages * 128, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T] * 500, device="cuda")
    out, lse = torch.full_like(q, 3.0), torch.full((T, N1), 3.0, device="cuda")
    P = bsa.params_for("TND", "PA_BBND", N1, N2)
    _, _, ws = bsa.bsa_decode(q, k, k.clone(), P, cu_seqlens_q=cu, seqused_kv=used, block_table=table, out=out, lse=lse)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN
    assert (out == 3).all() and (lse == 3).all()


@gpu
@pytest.mark.parametrize("T", [4, 500])  # rows that stream their own means, tiles
def test_select_overlapping_sequences(T):
    """Index rows belong to one sequence each, also where query tokens do not."""
    s = C.make(kvlens=(2000, 300, 1500), qlens=(T, 0, T + 1), N1=4, tail_rows=0, seed=18)
    s.qd[2][:2] = s.qd[0][-2:]
    s.q = torch.cat([s.qd[0], s.qd[2][2:]]).cuda()
    s.cu_q = torch.tensor([0, T, T - 2, 2 * T - 1], device="cuda")
    means = torch.randn(s.B, s.N2, s.NB, s.D, generator=s.g).to(s.dtype).cuda()
    index, ws = _select(s, means, dict(W=3))
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN
    assert torch.equal(_as_rows(s, index), C.ref_select(s, means, 3, "group").int())


@gpu
def test_select_overlapping_sequences_past_the_line():
    """128 sequences of all query tokens: 2^32 places for the rows that they
    need, of which the index has four."""
    T, N1, D, NB, W = 1 << 18, 32, 64, 65408, 5
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, N1, D, generator=g).to(BF).cuda().expand(T, N1, D)
    cu = torch.tensor([0, T] * 128, device="cuda")
    B = cu.shape[0] - 1
    means = torch.randn(1, 1, NB, D, generator=g).to(BF).cuda().expand(B, 1, NB, D)
    used = torch.full((B,), NB * 128, dtype=torch.int32, device="cuda")
    P = bsa.params_for("TND", "PA_BBND", N1, 1)
    index = torch.full((N1, 4, W), 77, dtype=torch.int16, device="cuda").view(torch.uint16)
    _, ws = bsa.bsa_select_blocks(q, means, P, cu_seqlens_q=cu, seqused_kv=used, index=index)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN | bsa.FLAG_BAD_INDEX
    best = (q[0].double() @ means[0, 0].double().T).topk(W, dim=1).indices.sort(dim=1).values
    assert torch.equal((index.to(torch.int32) & 0xFFFF), best.int().unsqueeze(1).expand(-1, 4, -1))


@gpu
def test_select_overlapping_sequences_past_32_bit_rows():
    """600 sequences of 2^30 - 128 query tokens (one row of memory): more than
    2^32 index rows, of which there are 2500, all of the first sequence."""
    T, D = (1 << 30) - 128, 64
    q = torch.ones(1, 1, D, dtype=BF, device="cuda").expand(T, 1, D)
    cu = torch.tensor([0, T] * 600, device="cuda")
    B = cu.shape[0] - 1
    means = torch.stack([torch.zeros(D), torch.ones(D)]).to(BF).cuda().expand(B, 1, 2, D)
    used = torch.full((B,), 128, dtype=torch.int32, device="cuda")
    used[0] = 256  # the other sequences have block 0 alone
    P = bsa.params_for("TND", "PA_BBND", 1, 1)
    index = torch.full((1, 2500, 1), 77, dtype=torch.int16, device="cuda").view(torch.uint16)
    _, ws = bsa.bsa_select_blocks(q, means, P, cu_seqlens_q=cu, seqused_kv=used, index=index)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN | bsa.FLAG_BAD_INDEX
    assert (index.to(torch.int32) == 1).all()


@gpu
def test_passes_and_decode_back_to_back():
    """Kernels that own an SM's tensor memory after one another in a stream."""
    s = C.make("TND", qlens=(300, 130), kvlens=(300, 130), N1=8, N2=2, tail_rows=0, poison=False)
    P = C.params(s, causal=True)
    k, v = s.k[:430].contiguous(), s.v[:430].contiguous()
    index = torch.full((s.N2, 5, 3), -1, dtype=torch.int16)
    for i in range(5):
        n = i + 1 if i < 3 else i - 2
        index[:, i, :n] = torch.arange(n, dtype=torch.int16)
    index = index.cuda().view(torch.uint16)
    kw = dict(cu_seqlens_q=s.cu_q, cu_seqlens_kv=s.cu_kv)
    outs = []
    for _ in range(20):
        o, l, _ = bsa.bsa_fwd(s.q, k, v, index, P, **kw)
        outs.append((o, l, bsa.bsa_decode(s.q, k, v, P, index=index, **kw)[:2]))
    torch.cuda.synchronize()
    o0, l0, (d0, e0) = outs[0]
    for o, l, (d, e) in outs:
        assert torch.equal(o, o0) and torch.equal(l, l0) and torch.equal(d, d0) and torch.equal(e, e0)
    C.check_decode(s, d0, e0, C.ref_decode(s, (index.to(torch.int32).cpu() & 0xFFFF).tolist(), causal=True))


# ------------------------------------------------------ flags of both kernels
FEW, TILES = dict(qlens=(1, 1), N1=4), dict(qlens=(40, 21), N1=8)  # rows of a kv head: 2; 160 and 84


@gpu
@pytest.mark.parametrize("kw", [FEW, TILES], ids=["few", "tiles"])
def test_decode_flags_of_both_kernels(kw):
    s = C.make(kvlens=(1000, 300), **kw, seed=23)
    T, ok = s.qlens[0], torch.isfinite
    n = s.qlens[0] + s.qlens[1]
    s.table[0, 3] = 1 << 20
    out, lse, ws = _decode(s, None, None, False)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_PAGE
    C.check_decode(s, out, lse, C.ref_decode(s, bad_pages=[(0, 3)]))
    rows = [[[0, 1, C.NONE], [0, 2, C.NONE]]] * s.N2  # the bad page is not among the selected
    out, lse, ws = _decode(s, rows, None, False)
    assert bsa.bsa_read_status(ws) == 0
    C.check_decode(s, out, lse, C.ref_decode(s, rows))
    for bad in ([0, 2, 3], [0, 2, 2], [0, 2, 1], [3, 0, 2], [C.NONE, 0, 60000]):  # of one row of one head
        mixed = [rows[0], [rows[0][0], bad]]
        out, lse, ws = _decode(s, mixed, None, False)
        assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX, bad
        C.check_decode(s, out, lse, C.ref_decode(s, mixed))
    out, lse, ws = _decode(s, [[[0, 1, 2]]] * s.N2, None, False)  # no row for the second sequence
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX
    assert (out[T:n] == 0).all() and torch.isneginf(lse[T:n]).all() and ok(lse[:T]).all()
    s.used[0] = s.table.shape[1] * s.page + 1
    out, lse, ws = _decode(s, None, None, False)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN
    assert (out[:T] == 0).all() and torch.isneginf(lse[:T]).all() and ok(lse[T:n]).all()


@gpu
@pytest.mark.parametrize("BKV", [128, 1024])
@pytest.mark.parametrize("kw", [FEW, TILES], ids=["few", "tiles"])
def test_decode_messy_index_is_flagged(kw, BKV):
    """Every row has an entry out of range, some behind all that are taken."""
    s = C.make(kvlens=(9000, 700), BKV=BKV, **kw, seed=29)
    rows = C.random_index(s, 40, s.N2, messy=True)
    out, lse, ws = _decode(s, rows, None, True)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX
    C.check_decode(s, out, lse, C.ref_decode(s, rows, causal=True))
    # a long valid row and one bad entry at its end
    nk = [-(-n // BKV) for n in s.kvlens]
    full = [[list(range(n)) + [C.NONE] * (80 - n) for n in nk] for _ in range(s.N2)]
    _, _, ws = _decode(s, full, None, True)
    assert bsa.bsa_read_status(ws) == 0
    full[-1][0][79] = nk[0]
    out, lse, ws = _decode(s, full, None, True)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_INDEX
    C.check_decode(s, out, lse, C.ref_decode(s, causal=True))


# ---------------------------------------------------------- many sequences
@gpu
@pytest.mark.parametrize("most", [3, 500])  # rows that stream their own means, tiles
@pytest.mark.parametrize("rows", ["group", "query"])
def test_select_many_sequences(most, rows):
    """More sequences than threads of a block, some of them empty."""
    g = torch.Generator().manual_seed(41)
    B = 600
    qlens = torch.randint(0, most + 1, (B,), generator=g)
    kvlens = torch.randint(0, 1500, (B,), generator=g)
    if most > 3:
        qlens += 150
    qlens[::7] = 0
    kvlens[::11] = 0
    s = C.make(kvlens=kvlens.tolist(), qlens=qlens.tolist(), N1=4, N2=2, D=64, seed=42, poison=False)
    R = sum(-(-n // s.BQ) for n in s.qlens)
    assert (R <= 2 * B) == (most == 3)
    means = torch.randn(s.B, s.N2, s.NB, s.D, generator=s.g).to(s.dtype).cuda()
    index, ws = _select(s, means, dict(W=4, rows=rows, sink=1))
    assert bsa.bsa_read_status(ws) == 0
    assert torch.equal(_as_rows(s, index), C.ref_select(s, means, 4, rows, sink=1).int())


@gpu
@pytest.mark.parametrize("kind", ["causal", "tree", "index"])
def test_decode_tiles_of_many_sequences(kind):
    """More sequences than threads of a block, through the 128-row tiles."""
    g = torch.Generator().manual_seed(43)
    B = 420
    qlens = torch.randint(0, 7, (B,), generator=g).tolist()
    kvlens = torch.randint(0, 300, (B,), generator=g).tolist()
    s = C.make(kvlens=kvlens, qlens=qlens, N1=8, N2=1, D=64, seed=44)
    tree = torch.cat([C.random_tree(T, 1, s.g) for T in qlens]) if kind == "tree" else None
    rows = C.random_index(s, 2, 1) if kind == "index" else None
    out, lse, ws = _decode(s, rows, tree, kind == "causal")
    assert bsa.bsa_read_status(ws) == 0
    C.check_decode(s, out, lse, C.ref_decode(s, rows, tree, kind == "causal"))


# --------------------------------------------- rows of more than 1024 blocks
def _wide(D, dtype, seed, T=(1, 130)):
    s = C.make(qlens=T, kvlens=(200, 200), N1=4, N2=2, D=D, dtype=dtype, seed=seed, poison=False)
    s.kvlens = [150000, 131073]  # lengths alone: no cache is read
    s.used = torch.tensor(s.kvlens, dtype=torch.int32, device="cuda")
    s.NB = 1172
    return s


@gpu
@pytest.mark.parametrize("D, dtype", [(128, FP), (64, BF), (128, BF)])
@pytest.mark.parametrize("W", [7, 400])
def test_select_wide_rows_with_forced_blocks(D, dtype, W):
    s = _wide(D, dtype, 51)
    means = torch.randn(s.B, s.N2, s.NB, D, generator=s.g).to(dtype).cuda()
    kw = dict(W=W, sink=3, local=2)
    index, ws = _select(s, means, kw)
    assert bsa.bsa_read_status(ws) == 0
    assert torch.equal(_as_rows(s, index), C.ref_select(s, means, W, "group", sink=3, local=2).int())


@gpu
@pytest.mark.parametrize("D, dtype", [(128, FP), (64, BF)])
@pytest.mark.parametrize("W", [7, 400])
def test_select_wide_rows_with_ties_beside_forced_blocks(D, dtype, W):
    """Equal means: hundreds of blocks are scored again, next to forced ones."""
    s = _wide(D, dtype, 52)
    for x in s.qd:
        x.copy_(x.sign())
    s.q = torch.cat(s.qd).cuda()
    means = torch.randn(s.B, s.N2, 1, D, generator=s.g).expand(s.B, s.N2, s.NB, D).clone()
    means[:, :, ::9] = torch.randn(s.B, s.N2, 1, D, generator=s.g)
    means = means.to(dtype).cuda()
    index, ws = _select(s, means, dict(W=W, sink=3, local=2))
    assert bsa.bsa_read_status(ws) == 0
    assert torch.equal(_as_rows(s, index), C.ref_select(s, means, W, "group", sink=3, local=2).int())


# ---------------------------------------------------------------- accuracy
@gpu
@pytest.mark.parametrize("T", [2, 40])  # tiles of 16 and of 128 rows
def test_decode_lse_of_a_dominant_key(T):
    """Two keys with scores 0 and -x: lse = log(1 + e^-x), small against 1.  The
    sum 1 + e^-x is rounded once (2^-24), e^-x is off by 2^-21 of itself
    (exponential) and x 2^-22 (products with log2 e in fp32), and the logarithm
    and its two products by 4 steps of the result."""
    D, N1 = 64, 8
    s = C.make(kvlens=(2,), qlens=(T,), N1=N1, N2=1, D=D, tail_rows=0, seed=61)
    s.k[s.table[0, 0].item(), :2] = 0
    s.k[s.table[0, 0].item(), 1, :, 0] = 1
    x = torch.linspace(3, 12, T * N1).view(T, N1).to(BF)
    s.q.zero_()
    s.q[..., 0] = -x.cuda()
    _, lse, _ = bsa.bsa_decode(s.q, s.k, s.v, C.params(s, scale=1.0), cu_seqlens_q=s.cu_q, **C.where(s))
    x = x.double()
    e = torch.exp(-x)
    want = torch.log1p(e)
    tol = 2.0 ** -24 + e * (2.0 ** -21 + x * 2.0 ** -22) + 4 * 2.0 ** -24 * want
    d = (lse.double().cpu() - want).abs()
    assert (d <= tol).all(), float((d / tol).max())


@gpu
def test_means_flag_only_pages_of_blocks_that_are_written():
    """A bad page behind the last block that the means have room for."""
    s = C.make(kvlens=(600, 500), qlens=(1, 1))
    s.table[0, 4] = -1
    small = torch.zeros(s.B, s.N2, 3, s.D, dtype=s.dtype, device="cuda")
    _, ws = bsa.bsa_block_means(s.k, C.params(s), **C.where(s), means=small)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN  # blocks left out, no page
    ref = C.ref_means(s)
    for b in range(2):
        m, mag = ref[b]
        d = (small[b].double().cpu() - m[:, :3]).abs()
        assert (d <= C.half_step(s.dtype) * m[:, :3].abs() + 2.0 ** -16 * mag[:, :3]).all()
    s.table[0, 2] = -1
    _, ws = bsa.bsa_block_means(s.k, C.params(s), **C.where(s), means=small)
    assert bsa.bsa_read_status(ws) == bsa.FLAG_BAD_SEQLEN | bsa.FLAG_BAD_PAGE
