"""The gated delta rule at the edges of what its calls allow: the default
stream by its handle, rows of no sequence in a new output, no value heads."""
from __future__ import annotations

import pytest
import torch

import test_gated_delta as td
from selective_scan_ss2d_b200 import binding

lib = td.lib   # the fixture: the built library


def test_backward_without_value_heads_is_refused(lib):
    """nothing would write dq and dk"""
    keep, p = td.ptr()
    assert td._bwd(lib, p, HK=1, H=0, vs=0) == -14
    assert td._bwd(lib, p, HK=0, H=0, qs=0, ks=0, vs=0) == 0
    assert td._fwd(lib, p, HK=1, H=0, vs=0) == 0   # an output of no heads


@pytest.mark.gpu
def test_default_stream_by_its_handle():
    """stream = 0 is the default stream, for a call's kernels and for the zeros of rows in no sequence"""
    t, _ = td.dev(td.make(1, 150, 1, 2, 32, 32), "bf16")
    do = torch.ones_like(t["v"])
    cu = torch.tensor([7, 60, 120], dtype=torch.int32).cuda()
    assert torch.cuda.default_stream().cuda_stream == 0
    want = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu)
    busy = [torch.cuda.Stream() for _ in range(64)]   # whatever other stream a call would use is behind
    torch.cuda.synchronize()
    for s in busy:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
    got = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu, stream=0)
    torch.cuda.synchronize()
    assert all(got[n] is None or torch.equal(got[n], want[n]) for n in want)


@pytest.mark.gpu
@pytest.mark.parametrize("L,cu", [(150, [7, 60, 120]), (150, [0, 149]), (150, [3]), (4, [1, 2]), (70, [70, 70])])
def test_rows_of_no_sequence_are_zero_in_a_new_output(L, cu):
    t, _ = td.dev(td.make(1, L, 1, 2, 32, 32), "bf16")
    for _ in range(4):   # what the allocator hands out next holds NaN
        torch.full_like(t["v"], float("nan"))
    o, _ = binding.gated_delta_rule_fwd(**t, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert not o[0, :cu[0]].any() and not o[0, cu[-1]:].any()
    assert bool(o[0, cu[0]:cu[-1]].any()) == (cu[-1] > cu[0])
