"""Calls of speculative decoding over the bf16 paged cache without a GPU: arguments that the checks let pass,
and a wait whose running out no GPU can show unless it has stopped answering."""
import ctypes
import os
import re

import pytest

from tests.test_spec_decode_host import CALLS, INV, ROOT, WS, X, lib  # noqa: F401 (lib: the fixture)


def _checked(lib, which, **change):
    """The status of a call whose workspace is too small, which is looked at last: WS if all else passes."""
    name, struct, good = CALLS[which]
    return getattr(lib, name)(ctypes.byref(struct(**{**good, **change})), X, 128, None)


APART = dict(k=64 * X, v=128 * X)


@pytest.mark.parametrize("change,status", [
    (dict(), WS), (dict(q_out=X), WS), (dict(q_out=X, q_stride=1024), INV),
    (dict(q_out=X, q_stride=1024, total_new=1), WS),  # a single row lies on itself
    (dict(q_out=X + 16, q_stride=1024, total_new=1), INV), (dict(q_out=X + 1024, q_stride=2048, total_new=1), WS),
    (dict(q_out=X + 16, total_new=1), INV), (dict(q_out=X, total_new=1), WS)], ids=lambda x: str(x))
def test_rotated_in_place(lib, change, status):  # noqa: F811
    assert _checked(lib, "append", **{**APART, **change}) == status


# five rows of 512 bytes of k and v, 1024 apart: 4608 bytes from 64 X and 128 X on; q_out takes 5120
@pytest.mark.parametrize("change,status", [
    (dict(q_out=64 * X), INV), (dict(q_out=128 * X), INV), (dict(q_out=64 * X - 5120), WS), (dict(q_out=64 * X - 5104), INV),
    (dict(q_out=128 * X + 4608), WS), (dict(q_out=128 * X + 4592), INV), (dict(q_out=64 * X + 512, total_new=1), WS),
    (dict(q_out=64 * X + 496, total_new=1), INV), (dict(q=None, q_out=64 * X), WS)], ids=lambda x: str(x))
def test_rotated_over_new_keys_and_values(lib, change, status):  # noqa: F811
    assert _checked(lib, "append", **{**APART, "k_stride": 512, "v_stride": 512, **change}) == status


def test_a_drain_that_runs_out_ends_the_scheduler():
    """The tree decode's scheduler leaves when the products have drained or the abort flag is raised, and has no limit of
    its own: whoever gives up waiting for the drain has to raise the flag (read in the source)."""
    with open(os.path.join(ROOT, "varlen_flashattention_gb300", "csrc", "decode_tree.cu")) as f:
        code = f.read()
    assert "if (given && ptx::warp_all(ptx::mbar_test(drain, 0))) break;" in code
    waits = re.findall(r"^.*mbar_wait\(drain,.*$", code, re.M)
    assert waits and all(re.search(r"if \(!ptx::mbar_wait\(drain,.*\) ctl->abort = 1;", w) for w in waits)
