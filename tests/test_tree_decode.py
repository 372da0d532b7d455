"""TreeDecode's own buffers, without a GPU: what a captured step keeps the addresses of stays where it is."""
import pytest
import torch

from paged_kv_cache_minmax_gb300 import build, kvmm
from paged_kv_cache_minmax_gb300.runtime import DecodeState, TreeDecode

B, N = 2, 4
CHAIN = [[-1, 0, 1, 2]] * B
FAN = [[-1, 0, 0, 0], [-1, 0, 0, 1]]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()


def trees(parent=CHAIN, dtype=torch.int32):
    k = torch.zeros(48, 16, 64, dtype=torch.bfloat16)
    st = DecodeState(B, 1, 4, 2, 64, 16, 12, 4, k, k.view(48, 64, 16), torch.zeros(B, 1, 2, 12, dtype=torch.int32),
                     torch.tensor([5, 40], dtype=torch.int32), device="cpu")
    return TreeDecode(st, torch.tensor(parent, dtype=dtype))


def held(t):
    return {n: getattr(t, n).data_ptr() for n in ("parent", "mask", "depth", "positions", "n_nodes", "tok_end")}


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_other_trees_go_where_the_first_were(dtype):
    t = trees(dtype=dtype)
    t.begin()
    at = held(t)
    t.set_trees(torch.tensor(FAN, dtype=dtype))
    t.begin(torch.tensor([4, 3], dtype=torch.int32))
    assert held(t) == at
    fresh = trees(FAN)
    fresh.begin(torch.tensor([4, 3], dtype=torch.int32))
    for n in ("parent", "mask", "depth", "positions", "n_nodes", "tok_end"):
        assert torch.equal(getattr(t, n), getattr(fresh, n)), n
    assert t.depth.tolist() == [[0, 1, 1, 1], [0, 1, 1, 2]]
    assert t.positions.tolist() == [[5, 6, 6, 6], [40, 41, 41, 42]]


def test_the_callers_tensor_is_not_kept():
    parent = torch.tensor(CHAIN, dtype=torch.int32)
    t = trees()
    t.set_trees(parent)
    parent.zero_()
    assert t.parent.tolist() == CHAIN


@pytest.mark.parametrize("shape", [(B, N + 1), (B, N - 1), (B + 1, N), (1, N), (B * N,), (N, B), (B, N, 1)])
def test_trees_of_another_shape_are_refused(shape):
    t = trees()
    t.begin()
    was = {n: getattr(t, n).clone() for n in ("parent", "mask", "depth", "positions")}
    with pytest.raises(ValueError, match="parent"):
        t.set_trees(torch.zeros(shape, dtype=torch.int32))
    t.begin()
    assert all(torch.equal(getattr(t, n), x) for n, x in was.items())


@pytest.mark.parametrize("parent", [[[-1, 0, 1]] * (B + 1), [[-1, 0, 1]], [-1, 0, 1]])
def test_a_state_of_another_batch_is_refused(parent):
    with pytest.raises(ValueError, match="parent"):
        trees(parent)


@pytest.mark.parametrize("wrong", [N, N + 1, 99, (1 << 31) - 1, 3, 2, -7, -(1 << 31)])
def test_impossible_parents_index_nothing(wrong):
    """A parent that is no earlier node: the node sees itself alone (below 0: itself and the root); the others are as
    they were.  (draft_verify reports it.)"""
    parent = [[-1, 0, wrong, 1], [-1, 0, 1, 2]]
    t = trees(parent)
    alone = 0b100 if wrong > 0 else 0b101
    assert t.mask.tolist() == [[0b1, 0b11, alone, 0b1011], [0b1, 0b11, 0b111, 0b1111]]
    assert t.depth.tolist() == [[0, 1, 0 if wrong > 0 else 1, 2], [0, 1, 2, 3]]
    assert torch.equal(kvmm.tree_masks(torch.tensor(parent)), t.mask)
