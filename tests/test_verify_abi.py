"""Refusals of dfc_verify_drafts through the C ABI, without a GPU, for calls
whose logits have no rows."""
import pytest

import lossless_entropy_coded_dfc_amd as dfc

pytest.importorskip("torch")
import test_serving_abi as abi  # noqa: E402


def test_no_rows_but_a_drafter_needs_a_workspace():
    # what was found for each request lies there, rows or none
    good = abi.Verify(2, 1000, 0, 2, None, 1000, 512, 1000, 256, None, None, None, 256, 512, 256, 1 << 20, None)
    size = abi.U64()
    f = dfc.library().dfc_verify_workspace
    f.argtypes = [abi.ctypes.POINTER(abi.Verify), abi.ctypes.POINTER(abi.U64)]
    assert f(good, abi.ctypes.byref(size)) == dfc.OK and size.value > 0
    abi.refused("dfc_verify_drafts", good, dfc.EINVAL, workspace_dev=None)
    abi.refused("dfc_verify_drafts", good, dfc.ESIZE, workspace_bytes=size.value - 1)
