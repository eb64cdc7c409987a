"""Argument checks of the routed experts in 8-bit floats that test_f8_host.py does not reach (no GPU)."""
from __future__ import annotations

import pytest

from tests.test_f8_host import E4, FP, I32, INV, _grad, _More, lib  # noqa: F401  (lib: the fixture)
from wna16_grouped_gemm_gb300 import f8


def test_sort_refuses_outputs_that_nothing_fills(lib):  # noqa: F811
    """Rows without x, scales without x and rows' scales without scales: refused, as the C ABI does, and not returned unwritten."""
    T, k, E, K = 4, 2, 8, 256
    ids, off, inv = _More(I32, T, k), _More(I32, E + 1), _More(I32, T, k)
    x, xs, rows, rs = _More(E4, T, K), _More(FP, T, 2), _More(E4, T * k, K), _More(FP, T * k, 2)
    for args, kw, message in (((None, ids, E), dict(rows=rows), "rows without x"),
                              ((None, ids, E), dict(scales=xs, row_scales=rs), "scales without x"),
                              ((None, ids, E), dict(row_scales=rs), "row_scales without scales"),
                              ((x, ids, E), dict(rows=rows, row_scales=rs), "row_scales without scales")):
        with pytest.raises(ValueError, match=message):
            f8.sort_tokens(*args, offsets=off, inv=inv, **kw)


def test_gradient_of_no_rows(lib):  # noqa: F811
    """Without rows (R = 0) there is no dy to write; with y or dweights the other one is still wanted where there are rows."""
    assert _grad(lib, R=0, y=None, w=None, dy=None, dw=None) == 0
    assert _grad(lib, R=0, y=None, dy=None, dw=None) == 0
    assert _grad(lib, R=1, y=None, dy=None, dw=None) == INV
    assert _grad(lib, R=1, dw=None) == INV


def test_gradient_of_nothing_is_refused(lib):  # noqa: F811
    d, inv = _More(FP, 4, 256), _More(I32, 4, 2)
    with pytest.raises(ValueError, match="neither dy nor y"):
        f8.unsort_tokens_grad(d, inv, want_dy=False)
