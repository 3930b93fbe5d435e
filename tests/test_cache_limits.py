"""The cache operators at the ends of what they accept: lengths that contradict
the storage, sizes near the limits, rules that switch kernels."""
import os
import shutil
import subprocess

import pytest
import torch

import block_sparse_variable_b200 as bsa
from tests import cache_cases as C
from tests.test_cache_ops import _decode

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
