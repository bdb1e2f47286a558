"""Calls of speculative decoding over the bf16 paged cache without a GPU: arguments that the checks let pass."""
import ctypes

import pytest

from tests.test_spec_decode_host import CALLS, INV, WS, X, lib  # noqa: F401 (lib: the fixture)


def _checked(lib, which, **change):
    """The status of a call whose workspace is too small, which is looked at last: WS if all else passes."""
    name, struct, good = CALLS[which]
    return getattr(lib, name)(ctypes.byref(struct(**{**good, **change})), X, 128, None)


@pytest.mark.parametrize("change,status", [
    (dict(), WS), (dict(q_out=X), WS), (dict(q_out=X, q_stride=1024), INV),
    (dict(q_out=X, q_stride=1024, total_new=1), WS),  # a single row lies on itself
    (dict(q_out=X + 16, q_stride=1024, total_new=1), INV), (dict(q_out=X + 1024, q_stride=2048, total_new=1), WS),
    (dict(q_out=X + 16, total_new=1), INV), (dict(q_out=X, total_new=1), WS)], ids=lambda x: str(x))
def test_rotated_in_place(lib, change, status):  # noqa: F811
    assert _checked(lib, "append", **change) == status
