"""The block operands' largest sizes: what a launch can hold is not refused, what it cannot is, without overflowing."""
import ctypes as C

import pytest
import torch

import token_dispatch_grouped_top_amd as mok

L = mok._lib
UNSUPPORTED, WIDEST = mok.MOK_ERR_UNSUPPORTED, (1 << 31) - 64


def quantise(rows, W, n=1, both=False):
    src = mok.mok_block8_source(0, 1, 16, 1 << 40, None, 0, 0, 0)
    return L.mok_block8_quantise(C.byref(src), rows, W, 16, n, 16, 16, *((16, 16) if both else (None, None)), 0, None)


def weights(n, N, K):
    return L.mok_block8_quantise_weights(16, 1, n, N, K, 16, 16, None, None, None)


def gemm(rows, K, N, n=1, out=1):
    return L.mok_block8_gemm(16, 16, rows, K, 16, n, 16, 16, N, 16, out, None)


def wgrad(rows, M, N, n=1):
    return L.mok_block8_wgrad(16, 16, M, 16, 16, N, rows, 16, n, 16, 0, 0, None)


@pytest.mark.parametrize("call", [
    lambda: quantise(1, WIDEST), lambda: quantise(1, WIDEST, both=True), lambda: quantise(1, 1 << 30, 2, both=True),
    lambda: quantise((1 << 31) - 1, 64), lambda: quantise((1 << 31) - 1, WIDEST),
    lambda: weights(1, 64, WIDEST), lambda: weights(1, WIDEST, 64), lambda: weights(1, WIDEST, WIDEST),
    lambda: weights(65535, WIDEST, WIDEST), lambda: weights(65535, 1024, 2176),
    lambda: gemm(1 << 24, 64, 8320), lambda: gemm(1, 64, WIDEST), lambda: gemm((1 << 30) + 1, 64, 64),
    lambda: gemm(1 << 20, 64, 1 << 17, out=0),
    lambda: wgrad(4, WIDEST, WIDEST, 256), lambda: wgrad(4, 1 << 15, 1 << 16, 129), lambda: wgrad((1 << 24) - 127, 64, 64)])
def test_too_large(call):
    assert call() == UNSUPPORTED


def test_largest_are_launched():
    """Without a GPU a call whose arguments pass ends with the launch's error; on one it would run."""
    if torch.cuda.is_available():
        pytest.skip("for a machine without a GPU")
    assert quantise(1, (1 << 30) - 128) == mok.MOK_ERR_HIP
    assert weights(127, 32768, 32768) == mok.MOK_ERR_HIP
    assert gemm(1 << 24, 64, 7168) == mok.MOK_ERR_HIP         # 2^18 tiles of rows, 56 of columns
    assert gemm(1100000, 64, 8192) == gemm(1100000, 64, 8192, out=0) == mok.MOK_ERR_HIP
    assert gemm((1 << 30) - 64, 64, 64) == mok.MOK_ERR_HIP
    assert wgrad(4, 1 << 15, 1 << 16, 127) == mok.MOK_ERR_HIP
