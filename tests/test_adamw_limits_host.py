"""Host checks of the largest list of the AdamW step: a launch has 2^24 - 1
workgroups, each of one unit of a tensor, for each state format."""
import ctypes as C

import pytest

import token_dispatch_grouped_top_amd as mok

UNITS = (1 << 24) - 1
SIZE = {mok.MOK_STATE_F32: 1024, mok.MOK_STATE_MXFP8: 2048}       # elements of a unit


def _build(*tensors):
    """Status for (format, elements) tensors with a table of no bytes: MOK_ERR_WORKSPACE where all else is right."""
    a = (mok.mok_adamw_tensor * len(tensors))(*(
        mok.mok_adamw_tensor(p=(i + 1) << 50, grad=1 << 20, m=2 << 20, v=3 << 20, m_scale=64, v_scale=64, n=n,
                             state_format=fmt, lr_scale=1.0) for i, (fmt, n) in enumerate(tensors)))
    return mok._lib.mok_adamw_build_table(a, len(a), 64, 0, C.byref(mok.mok_adamw_plan()), None)


@pytest.mark.parametrize("fmt", sorted(SIZE))
def test_largest_list_of_one_format(fmt):
    size, other = SIZE[fmt], 1 - fmt
    fits, not_fits = mok.MOK_ERR_WORKSPACE, mok.MOK_ERR_UNSUPPORTED
    assert _build((fmt, UNITS * size)) == fits
    assert _build((fmt, UNITS * size + 1)) == not_fits
    assert UNITS % 3 == 0
    assert _build(*[(fmt, UNITS // 3 * size)] * 3) == fits
    assert _build(*[(fmt, UNITS // 3 * size)] * 3, (fmt, 1)) == not_fits
    assert _build(*[(fmt, UNITS // 3 * size)] * 2, (fmt, (UNITS // 3 - 1) * size + 1)) == fits   # a last unit of one element
    assert _build((fmt, UNITS * size), (other, UNITS * SIZE[other])) == fits                      # a launch for each
    assert _build((fmt, 1 << 62)) == not_fits
    assert _build(*[(fmt, UNITS * size)] * 2) == not_fits
