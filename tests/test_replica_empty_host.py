"""Workspace queries of empty batches, as a caller makes them before the call."""
import ctypes

import pytest

from test_replica_ops_host import Z, lib  # noqa: F401


@pytest.mark.parametrize("rows,cols", [(0, 64), (0, 4096), (0, 50000), (5, 0), (4, 0), (0, 0)])
def test_nothing_needs_no_workspace(lib, rows, cols):  # noqa: F811
    for query in (lib.vrcclRmsNormWorkspace, lib.vrcclLayerNormWorkspace):
        n = Z(77)
        assert query(rows, cols, ctypes.byref(n)) == 0 and n.value == 0, query.__name__
