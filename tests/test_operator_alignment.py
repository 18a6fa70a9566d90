"""Pointers off their elements are refused by the expert-order moves, the
router's gradient and the dense product (CPU: every call here returns before a
kernel could launch)."""
import ctypes as C

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def milo():
    import int3_gemm_rank_b200 as m
    m.lib()
    return m


F = C.c_void_p(0x10000)
OFF = [C.c_void_p(0x10001), C.c_void_p(0x10002)]         # no address of a 32-bit element


def calls(L, bad):
    """(name, call with pointer `bad` in one place) of every 32-bit operand."""
    def put(n):
        for i in range(n):
            yield [bad if i == j else F for j in range(n)]

    for inv, w, st in put(3):
        yield "milo_dispatch", L.milo_dispatch(F, 1, 4, 2, 64, inv, w, F, 1, st, None)
        yield "milo_combine", L.milo_combine(F, 1, 4, 2, 64, inv, w, None, F, 1, st, None)
    for inv, w, dw, st in put(4):
        yield "milo_dispatch_backward", L.milo_dispatch_backward(F, 1, 4, 2, 64, inv, w, F, F, 1, dw, st, None)
        yield "milo_combine_backward", L.milo_combine_backward(F, 1, 4, 2, 64, inv, w, F, F, 1, dw, st, None)
    for ids, w, dw, st in put(4):
        yield "milo_route_backward", L.milo_route_backward(F, ids, w, dw, 4, 8, 2, 0, F, 0, st, None)
    yield "milo_dense_linear", L.milo_dense_linear(F, F, 1, 4, 16, 64, None, None, 0, F, 1, None, bad, None)
    yield "milo_dense_linear_backward", L.milo_dense_linear_backward(F, 1, F, F, 1, 4, 16, 64, 0, None, F, F, F, F, 1 << 30,
                                                                     bad, None)


@pytest.mark.parametrize("bad", OFF)
def test_32_bit_operands_off_their_elements(milo, bad):
    for name, status in calls(milo.lib(), bad):
        assert status == milo.MILO_ERR_INVALID_ARG, name
        assert "aligned" in milo.lib().milo_last_error().decode(), name


def test_logits_off_their_elements(milo):
    L = milo.lib()
    assert L.milo_route_backward(OFF[0], F, F, F, 4, 8, 2, 0, F, 0, None, None) == milo.MILO_ERR_INVALID_ARG
