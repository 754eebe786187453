"""Offsets outside the contract: whatever cu_seqlens holds, no row outside the call's own
[0, total) is a new token.  The arithmetic on the CPU first, then the kernels, which may
write nothing beyond their outputs."""
import ctypes
import itertools
import os
import subprocess

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm

INT_MIN, INT_MAX = -(2**31), 2**31 - 1


@pytest.fixture(scope="module")
def seq_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("seq")
    csrc = os.path.join(os.path.dirname(fa.__file__), "csrc")
    src, so = str(d / "seq.cpp"), str(d / "seq.so")
    with open(src, "w") as f:
        f.write('#include "paged_seq.h"\nextern "C" void seq(int a, int b, int len, int total, int most, int places, int *o) {'
                ' const fa::PagedSeq s = fa::paged_seq_of(a, b, len, total, most, places);'
                ' o[0] = s.start; o[1] = s.n; o[2] = s.len; o[3] = s.keys; }\n')
    # -ftrapv: a 32-bit sum or difference that overflows ends the child process
    subprocess.run(["g++", "-O1", "-ftrapv", "-std=c++17", "-shared", "-fPIC", f"-I{csrc}", src, "-o", so], check=True)
    f = ctypes.CDLL(so).seq
    out = (ctypes.c_int * 4)()

    def call(*a):
        f(*a, out)
        return tuple(out)

    return call


def test_no_offsets_leave_the_arrays(seq_of):
    ends = [INT_MIN, INT_MIN + 1, -(2**30), -257, -1, 0, 1, 2, 5, 6, 7, 2**30, INT_MAX - 1, INT_MAX]
    lens = [INT_MIN, -1, 0, 3, 2**30 - 1, 2**30, INT_MAX]
    for c0, c1, n, total, most, places in itertools.product(ends, ends, lens, [0, 1, 6, INT_MAX], [1, 3, 256],
                                                            [16, 2**30]):
        start = min(max(c0, 0), total)
        new = min(max(min(c1, total) - start, 0), most)
        cached = min(max(n, 0), places)
        got = seq_of(c0, c1, n, total, most, places)
        assert got == (start, new, cached, min(cached + new, places)), (c0, c1, n, total, most, places)
        assert got[0] + got[1] <= total


TABLES = [[0, INT_MIN, 6, 6], [6, INT_MIN, INT_MIN, INT_MIN], [INT_MIN, INT_MAX, INT_MIN, INT_MAX], [5, 2, -3, 6],
          [3, INT_MIN + 1, 4, INT_MIN], [INT_MAX, INT_MIN, -1, INT_MAX], [-7, -2, 2, 9]]


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d,most,tree", [(2, 2, 128, 3, True), (4, 1, 64, 4, False), (4, 1, 128, 6, True),
                                               (32, 1, 64, 6, True), (64, 1, 128, 6, False), (8, 2, 256, 6, True)])
def test_offsets_outside_the_contract_write_nothing_outside(H, Hkv, d, most, tree):
    s = pm.Setup([40, 7, 100], [2, 2, 2], 16, Hkv, d, seed=d, H=H)
    guard = 300  # more rows than max_new on either side
    for cu in TABLES:
        o = torch.full((6 + 2 * guard, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2 * guard + 6, H), 7.0, device="cuda").view(-1)  # [H, 6] in the middle
        mid = lse[guard * H : (guard + 6) * H].view(H, 6)
        mask = torch.full((6, 1), -1, dtype=torch.int64, device="cuda") if tree else None
        t_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, t_cu, most, tree_mask=mask,
                               out=o[guard : guard + 6], lse=mid)
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == fa.FA_OK, cu
        assert (o[:guard] == 7).all() and (o[guard + 6 :] == 7).all(), cu
        assert (lse[: guard * H] == 7).all() and (lse[(guard + 6) * H :] == 7).all(), cu
        mine = set()  # rows that belong to some sequence; the others are left alone
        for c0, c1 in zip(cu, cu[1:]):
            a = min(max(c0, 0), 6)
            mine |= set(range(a, a + min(max(min(c1, 6) - a, 0), most)))
        for t in set(range(6)) - mine:
            assert (o[guard + t] == 7).all() and (mid[:, t] == 7).all(), (cu, t)
