"""Outputs of the serving operators over their inputs: refused on the host,
element by element (no GPU)."""
import ctypes
import itertools

import pytest
import torch

import dual_scale_solver_b200 as dq
from dual_scale_solver_b200 import serving

ARG, CUDA = -1, -6
BASE = 1 << 20                              # an address, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    from dual_scale_solver_b200 import build
    build.build()


def _status(call, refused):
    """A call that is not refused reaches the device, which is not there."""
    if not refused and torch.cuda.is_available():
        return CUDA
    return call()


def _elements(at, token, head, tokens, heads, dim):
    return {at + t * token + h * head + d for t in range(tokens) for h in range(heads) for d in range(dim)}


def _norm(res, out, stride, out_stride, x=BASE + (1 << 22)):
    f, p = dq.format_preset("mxfp4"), lambda e: None if e is None else ctypes.c_void_p(BASE + 2 * e)  # noqa: E731
    return serving._lib().dq_add_rmsnorm_quant(ctypes.c_void_p(x), 64, p(res), stride, ctypes.c_void_p(BASE + (1 << 23)),
                                               1, None, 1e-5, 3, 64, ctypes.byref(f), p(out), out_stride,
                                               ctypes.c_void_p(BASE + (1 << 24)), ctypes.c_void_p(BASE + (1 << 25)), None)


@pytest.mark.parametrize("stride", [64, 72, 128, 192])
def test_norm_residual_out_over_an_input(stride):
    base = 4096
    for shift in range(-4 * stride, 4 * stride + 1, 8):
        a, b = _elements(base, stride, 0, 3, 1, 64), _elements(base + shift, stride, 0, 3, 1, 64)
        refused = shift != 0 and bool(a & b)
        want = ARG if refused else CUDA
        assert _status(lambda: _norm(base, base + shift, stride, stride), refused) == want, shift
        # over x
        if stride == 64:
            assert _status(lambda: _norm(None, base + shift, stride, stride, x=BASE + 2 * base), refused) == want, shift
    # other strides: apart or refused
    assert _norm(base, base + 64, 128, 64) == ARG
    assert _norm(base, base + 2 * 128 + 56, 128, 64) == ARG
    assert _status(lambda: _norm(base, base + 2 * 128 + 64, 128, 64), False) == CUDA
    assert _status(lambda: _norm(base + 2 * 64 + 64, base, 128, 64), False) == CUDA
    # in place over one input, and over a part of the other
    assert _norm(base + 8, base, 64, 64, x=BASE + 2 * base) == ARG
    assert _status(lambda: _norm(base, base, 64, 64, x=BASE + 2 * base), False) == CUDA


LAYOUTS = [(256, 128), (128, 3 * 128), (512, 128), (384, 192), (512, 256)]     # (token, head), 3 x 2 rows of 128


def _places():
    return (serving.dq_kv_cache(BASE, BASE, BASE, BASE, 8, 16, 2, 128),
            serving.dq_kv_batch(BASE, BASE, BASE, 2, 4, 4))


def _read(at, other, a, b):
    f, (c, m) = dq.format_preset("mxfp4"), _places()
    p = lambda e: ctypes.c_void_p(BASE + 2 * e)                # noqa: E731
    return serving._lib().dq_kv_read(p(at), *a, p(other), *b, 3, ctypes.addressof(c), ctypes.addressof(m),
                                     ctypes.byref(f), None)


def _check_pairs(call):
    base = 8192
    for a, b in itertools.product(LAYOUTS, LAYOUTS):
        one, end = _elements(base, *a, 3, 2, 128), base + 2 * a[0] + a[1] + 128
        for shift in range(-1600, 1601, 40):
            other = _elements(base + shift, *b, 3, 2, 128)
            meet = base + shift < end and base < base + shift + 2 * b[0] + b[1] + 128
            refused = bool(one & other) if a == b else meet
            assert refused or not (one & other)
            want = ARG if refused else CUDA
            assert _status(lambda: call(base, base + shift, a, b), refused) == want, (a, b, shift)


def test_read_keys_over_values():
    _check_pairs(_read)
    assert _read(8192, 8192, (256, 128), (512, 128)) == ARG


def _attend(at, other, a, b, tokens=3):
    f, (c, m) = dq.format_preset("mxfp4"), _places()
    p = lambda e: ctypes.c_void_p(BASE + 2 * e)                # noqa: E731
    return serving._lib().dq_kv_attention(p(at), *a, p(other), *b, tokens, 2, 0.1, 1, ctypes.addressof(c),
                                          ctypes.addressof(m), ctypes.byref(f), ctypes.c_void_p(BASE), 1 << 30, None)


def test_attention_over_its_queries():
    _check_pairs(_attend)
    # queries that are all one row
    assert _attend(8192, 8192 + 120, (0, 0), (256, 128)) == ARG
    assert _attend(8192, 8192 - 512 - 128, (0, 0), (256, 128)) == ARG
    assert _status(lambda: _attend(8192, 8192 + 128, (0, 0), (256, 128)), False) == CUDA
    # one token: its stride does not matter
    assert _status(lambda: _attend(8192, 8192 + 128, (1024, 256), (256, 256), tokens=1), False) == CUDA
    assert _attend(8192, 8192 + 256, (1024, 256), (256, 256), tokens=1) == ARG
