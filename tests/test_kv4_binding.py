"""What the Python binding of the rotated appends checks and hands on, without a GPU: tensors that only say that they
are on one."""
import ctypes

import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm


class OnDevice(torch.Tensor):
    """A CPU tensor that passes for one on device 0."""

    is_cuda = True

    def get_device(self):
        return 0


def here(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


B, N, HQ, HKV, D = 3, 4, 8, 2, 64


def arguments(rope=None, q_out=None, n=N):
    """What _append_rows makes of n new rows of B sequences."""
    f = (B, 1, HQ, HKV, D)
    tok = here(B, dtype=torch.int32)
    return kvmm._append_rows(f, here(B, n, HQ, D), here(B, n, HKV, D), here(B, n, HKV, D), tok, tok, rope,
                             here(B, n, HQ, D) if q_out is None else q_out, 0)


def turn(positions=None):
    return kvmm.Rope(here(9, 2, D // 2, dtype=torch.float32), D, positions=positions)


def ints(*shape):
    return here(*shape, dtype=torch.int32)


# ---- positions are [B][n_new] ---------------------------------------------------------------------------------
@pytest.mark.parametrize("shape", [(B, N), (B + 2, N), (B * N,), (B * N + 5,), (1, B * N), (B * N, 1), (B, N, 1)])
def test_positions_that_are_dense_rows_pass(shape):
    pos = ints(*shape)
    assert arguments(turn(pos))[6] is not None


@pytest.mark.parametrize("shape", [(B, N + 1), (B, 2 * N), (N, B), (B, 1), (B, 2, N), (B - 1, N), (B * N - 1,)])
def test_positions_of_other_rows_are_refused(shape):
    """A wider or otherwise laid out tensor has its rows where the kernel does not look for them."""
    with pytest.raises(ValueError, match="positions"):
        arguments(turn(ints(*shape)))


# ---- so is q_out ----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n,shape", [(N, (B, N, HQ, D)), (N, (B + 1, N, HQ, D)), (N, (B * N * HQ * D + 64,)), (1, (B, HQ, D)),
                                     (1, (B, 1, HQ, D)), (1, (B + 4, HQ, D)), (N, (B, N, HQ * D)), (N, (B * N, HQ, D))])
def test_q_out_of_dense_rows_passes(n, shape):
    assert arguments(q_out=here(*shape), n=n)[7] is not None


@pytest.mark.parametrize("n,shape", [(N, (B, N + 1, HQ, D)), (N, (B, N, HQ + 1, D)), (N, (B, N, HQ, 2 * D)), (1, (B, 2, HQ, D)),
                                     (N, (B, HQ, N, D)), (1, (B, HQ, 2 * D)), (1, (B, 2 * HQ, D))])
def test_q_out_of_other_rows_is_refused(n, shape):
    with pytest.raises(ValueError, match="q_out"):
        arguments(q_out=here(*shape), n=n)


# ---- a rope's tensors -----------------------------------------------------------------------------------------
def handed_on(rope):
    """The struct that a call with this rope gets."""
    return ctypes.cast(arguments(rope)[6], ctypes.POINTER(kvmm.RopeStruct)).contents


def test_positions_may_be_replaced():
    """The pointer handed on is that of the tensor that was checked."""
    rope = turn()
    assert rope.positions is None and handed_on(rope).positions is None
    for pos in (ints(B, N), ints(B, N), None, ints(B * N)):
        rope.positions = pos
        assert rope.positions is pos
        assert handed_on(rope).positions == (None if pos is None else pos.data_ptr())
    for bad, error in ((torch.zeros(B, N, dtype=torch.int32), "CUDA"), (here(B, N, dtype=torch.int64), "int32"),
                       (ints(N, B).t(), "contiguous")):
        with pytest.raises(ValueError, match=error):
            rope.positions = bad
    assert rope.positions is pos  # a refused tensor changes nothing
    assert handed_on(rope).positions == pos.data_ptr()


def test_the_table_stays():
    rope = turn()
    for name, value in (("table", here(9, 2, D // 2, dtype=torch.float32)), ("dim", 32)):
        with pytest.raises(AttributeError):
            setattr(rope, name, value)
    assert handed_on(rope).table == rope.table.data_ptr() and rope.dim == D
