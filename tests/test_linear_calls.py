"""Calls of the BF16 layers that are refused, by the C entry points and in Python: no GPU."""
import pytest

import sgemm_row_major_gb300 as sg
from test_linear_refusals import FAKE, kept, lib, refused  # noqa: F401 (fixture)

WIDE = 1 << 31  # a row stride that is not supported


def test_kept_rows_too_far_apart(lib):  # noqa: F811
    """A kept matrix whose row stride is too large is as unsupported as any other, and one that is not read is not looked at."""
    unsupported = sg.STATUS["ERR_UNSUPPORTED"]
    for scale in (None, FAKE):
        far, near = kept(ld=WIDE, scale=scale), kept(ld=16, scale=scale)
        layer = (4, 8, 16, FAKE, 8, FAKE, 8, FAKE, 2, FAKE, 16, near, FAKE, 16, 1, None)
        refused(lib.sgemm_linear, layer, [(unsupported, {12: far})], empty=[{1: 0, 12: far}])
        gated = (4, 8, 16, FAKE, 8, FAKE, 8, FAKE, 8, 2, near, near, FAKE, 16, None)
        refused(lib.sgemm_gated, gated, [(unsupported, {11: far}), (unsupported, {12: far})])
        grad = (4, 8, 16, FAKE, 16, kept(ld=8, scale=scale), FAKE, 8, 2, near, FAKE, 8, FAKE, 8, 1, FAKE, None)
        refused(lib.sgemm_linear_backward, grad, [(unsupported, {6: far}), (unsupported, {10: far}), (-6, {6: kept(ld=7, scale=scale)})],
                empty=[{6: far, 10: far, 9: 0, 11: None, 13: None, 16: None}])
        grad = (4, 8, 16, FAKE, 16, kept(ld=8, scale=scale), FAKE, 8, FAKE, 8, 2, near, near, FAKE, 8, FAKE, 8, FAKE, 8, 1, FAKE, 16, None)
        refused(lib.sgemm_gated_backward, grad, [(unsupported, {6: far}), (unsupported, {12: far}), (unsupported, {13: far}), (-12, {12: kept(ld=15, scale=scale)})],
                empty=[{6: far, 14: None, 16: None, 18: None, 21: None}])
