"""A bounded wait of the weight sums' kernel, made to run out on the GPU: block 0 leaves out one
barrier arrival, the kernel comes back with FA_ERR_TIMEOUT (after 2 ms in this build), and the
next call in the same process is correct.  Nothing here faults the GPU."""
import ctypes
import os
import re

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
from exact_attention_blackwell_gb300 import build

CSRC = os.path.join(os.path.dirname(fa.__file__), "csrc")


@pytest.mark.parametrize("source", ["fa_rope.cu", "fa_weights.cu", "fa_evict.cu"])
def test_early_kernels_promise_no_constant_contents(source):
    text = open(os.path.join(CSRC, source)).read()
    bodies = re.split(r"__global__", text)[1:]
    assert bodies
    for body in bodies:
        assert "__restrict__" not in body and "grid_wait();" in body and "__ldg" not in body


@pytest.fixture(scope="module")
def stall_lib(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("stall") / "libfa_stall.so")
    build.build(force=True, extra_flags=["-DFA_TEST_STALL", "-DFA_WAIT_LIMIT_NS=2000000ull"], lib_path=path)
    lib = ctypes.CDLL(path)
    for name in ("fa_attention_weights_paged", "fa_last_device_status", "fa_last_device_status_site", "fa_debug_stall"):
        getattr(lib, name).restype, getattr(lib, name).argtypes = fa.SIGNATURES[name]
    return lib


@pytest.mark.gpu
@pytest.mark.slow
@pytest.mark.parametrize("new,H,Hkv,d", [(1, 4, 4, 128), (70, 8, 2, 128), (20, 2, 1, 64), (9, 16, 1, 256), (1, 2, 2, 256)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_correct(stall_lib, new, H, Hkv, d):
    s = pm.Setup([4000] * 2, [new] * 2, 64, Hkv, d, seed=d, H=H)
    _, lse = fa.attention_fwd_paged(s.q, s.k_pages, s.v_pages, s.t_table, s.t_lens, s.t_cu, new)
    many = 100  # the two sequences again and again, so that block 0 has more tiles than its buffers hold
    table, lens, q = s.t_table.repeat(many, 1), s.t_lens.repeat(many), s.q.repeat(many, 1, 1)
    cu, many_lse = torch.arange(2 * many + 1, dtype=torch.int32, device="cuda") * new, lse.repeat(1, many)

    def run(B, table, lens, cu, q, lse):
        w = torch.zeros((B, Hkv, 4300), device="cuda")
        assert stall_lib.fa_attention_weights_paged(
            q.data_ptr(), s.k_pages.data_ptr(), table.data_ptr(), lens.data_ptr(), cu.data_ptr(), None, 0, lse.data_ptr(),
            w.data_ptr(), 4300, 1.0, B, s.cols, s.num_pages, s.page, new, q.shape[0], H, Hkv, d, d**-0.5, None) == fa.FA_OK
        return w

    want = torch.zeros((2, Hkv, 4300), device="cuda")
    fa.attention_weights_paged(s.q, s.k_pages, s.t_table, s.t_lens, s.t_cu, new, lse, want)
    torch.cuda.synchronize()
    site = ctypes.c_int(-1)
    assert stall_lib.fa_last_device_status_site(None, ctypes.byref(site)) == fa.FA_OK and site.value == 0
    assert stall_lib.fa_debug_stall(6) == fa.FA_OK
    try:
        run(2 * many, table, lens, cu, q, many_lse)
        st = stall_lib.fa_last_device_status_site(None, ctypes.byref(site))
    finally:
        assert stall_lib.fa_debug_stall(0) == fa.FA_OK
    assert st == fa.FA_ERR_TIMEOUT and 43 <= site.value <= 51, (st, site.value)
    got = run(2, s.t_table, s.t_lens, s.t_cu, s.q, lse)
    torch.cuda.synchronize()
    assert stall_lib.fa_last_device_status(None) == fa.FA_OK
    assert torch.equal(got, want)
