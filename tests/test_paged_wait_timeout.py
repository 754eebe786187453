"""Bounded waits of the paged attention kernels, made to run out on the GPU: block 0
leaves out one barrier arrival that nothing else gives, the kernel comes back with
FA_ERR_TIMEOUT, and the next call in the same process is correct.  Nothing here
faults the GPU: the waits end by themselves (after 2 ms in this build)."""
import ctypes

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
from exact_attention_blackwell_gb300 import build

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

# waits that can run out first: the one for the missing signal, or one that began before it
SITES = {4: {34, 35, 36}, 5: {42, 41}}


@pytest.fixture(scope="module")
def stall_lib(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("stall") / "libfa_stall.so")
    build.build(force=True, extra_flags=["-DFA_TEST_STALL", "-DFA_WAIT_LIMIT_NS=2000000ull"], lib_path=path)
    lib = ctypes.CDLL(path)
    for name in ("fa_fwd_paged", "fa_fwd_paged_workspace_bytes", "fa_last_device_status", "fa_last_device_status_site",
                 "fa_debug_stall"):
        getattr(lib, name).restype, getattr(lib, name).argtypes = fa.SIGNATURES[name]
    return lib


def run(lib, s, H, max_new):
    o = torch.empty_like(s.q)
    lse = torch.empty((H, s.total), device="cuda")
    nb = lib.fa_fwd_paged_workspace_bytes(s.B, max_new, H, s.Hkv, s.d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    assert lib.fa_fwd_paged(s.q.data_ptr(), s.k_pages.data_ptr(), s.v_pages.data_ptr(), s.t_table.data_ptr(),
                            s.t_lens.data_ptr(), s.t_cu.data_ptr(), None, 0, o.data_ptr(), lse.data_ptr(), s.B, s.cols,
                            s.num_pages, s.page, max_new, s.total, H, s.Hkv, s.d, s.d**-0.5, ws.data_ptr(), nb,
                            None) == fa.FA_OK
    return o, lse


# a few long rows of the table each, so that block 0 has more tiles than its ring holds
@pytest.mark.parametrize("mode,new,H,Hkv,d", [(4, 70, 4, 2, 128), (4, 20, 2, 1, 64), (4, 9, 4, 1, 256), (4, 20, 4, 4, 128),
                                              (5, 1, 4, 4, 128), (5, 2, 2, 1, 64), (5, 3, 4, 2, 256)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_correct(stall_lib, mode, new, H, Hkv, d):
    s = pm.Setup([1500] * 3, [new] * 3, 64, Hkv, d, seed=mode + d, H=H)
    lens = torch.full((300,), 1500, dtype=torch.int32, device="cuda")
    wide = pm.Setup([0], [1], 16, 1, 64, seed=1, H=1)
    wide.__dict__.update(s.__dict__)
    wide.B, wide.total = 300, 300 * new  # one hundred times the three sequences
    wide.t_table, wide.t_lens = s.t_table.repeat(100, 1).contiguous(), lens
    wide.t_cu = torch.arange(301, dtype=torch.int32, device="cuda") * new
    wide.q = s.q.repeat(100, 1, 1)
    site = ctypes.c_int(-1)
    assert stall_lib.fa_last_device_status_site(None, ctypes.byref(site)) == fa.FA_OK and site.value == 0
    assert stall_lib.fa_debug_stall(mode) == fa.FA_OK
    try:
        run(stall_lib, wide, H, new)
        st = stall_lib.fa_last_device_status_site(None, ctypes.byref(site))
    finally:
        assert stall_lib.fa_debug_stall(0) == fa.FA_OK
    assert st == fa.FA_ERR_TIMEOUT and site.value in SITES[mode], (st, site.value)
    o, lse = run(stall_lib, s, H, new)
    torch.cuda.synchronize()
    assert stall_lib.fa_last_device_status(None) == fa.FA_OK
    pm.check_attention(s, o, lse, pm.attention(s, s.q), f"after stall mode {mode}")
