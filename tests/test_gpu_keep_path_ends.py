"""kv_keep_path: rows that stay where they are have a place too, or are told."""
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from tests.test_gpu_keep_path import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("meta", [True, False])
@pytest.mark.parametrize("T", [16, 32])
@pytest.mark.parametrize("seq,path,beyond", [(61, [0, 1, 2], False), (62, [0, 1, 2], True), (64, [0], True), (63, [0], False),
                                             (64, [], False), (60, [0, 1, 2, 3, 4, 5], True), (62, [0, 1, 4], True),
                                             (50, list(range(14)), False), (50, list(range(15)), True)])
def test_a_prefix_beyond_the_table(meta, T, seq, path, beyond):
    c = Case([seq, 3], [path, [0, 2]], 15, T=T, Pmax=64 // T, seed=seq)
    if not meta:
        c.call(meta=None)
        torch.cuda.synchronize()
        assert int(c.err) == (kvmm.ERR_OUT_OF_RANGE if beyond else 0)
        c.err.zero_()
        c.k_pool.copy_(c.before[0])
        c.v_pool.copy_(c.before[1])
    c.call()
    c.check(err=kvmm.ERR_OUT_OF_RANGE if beyond else 0)


@pytest.mark.parametrize("entry", [-1, 1 << 30])
@pytest.mark.parametrize("page,path,told", [(2, [0, 1], True), (3, [0, 1], False), (3, list(range(9)), True), (2, [], False), (4, [0, 9], False)])
def test_rows_that_stay_in_a_page_without_a_place(entry, page, path, told):
    """No bounds are kept: the rows alone ask for their pages."""
    c = Case([40], [path], 14, L=1, seed=9, Pmax=6)
    c.table[0, 0, :, page] = entry
    c.call(meta=None)
    torch.cuda.synchronize()
    assert int(c.err) == ((kvmm.ERR_NULL_BLOCK if entry < 0 else kvmm.ERR_OUT_OF_RANGE) if told else 0)
