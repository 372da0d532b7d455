"""The plain forms of speculative decoding, against their definitions and against sampling theory (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import build, kvmm
from tests import tree_plain


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return kvmm.load()


# ---- masks ----------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 2, 7, 63, 64])
def test_tree_masks(n):
    r = np.random.RandomState(n)
    parent = np.full((3, n), -1)
    for i in range(1, n):
        parent[:, i] = [i - 1, r.randint(0, i), 0]
    got = kvmm.tree_masks(torch.from_numpy(parent).to(torch.int32)).numpy().view(np.uint64)
    assert np.array_equal(got, tree_plain.masks(parent))
    assert np.array_equal(got[0], [(1 << (i + 1)) - 1 for i in range(n)])


@pytest.mark.parametrize("shape", [(3,), (2, 65), (2, 0), (1, 2, 3)])
def test_tree_masks_refuses(shape):
    with pytest.raises(ValueError, match="parent"):
        kvmm.tree_masks(torch.zeros(*shape, dtype=torch.int32))


# ---- verification ---------------------------------------------------------------------------------------------
def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("kind", ["rows", "distinct", "certain"])
def test_the_first_token_is_distributed_as_the_target(kind):
    """Whatever the draft proposes, the token behind the root follows the target's row: 20,000 walks over 6 tokens, a
    chi-square of 5 degrees of freedom below 25.7 (1e-4)."""
    r = np.random.RandomState(11)
    V, n, rounds = 6, 4, 20000
    target, draft = softmax(r.randn(n, V) * 1.2), softmax(r.randn(n, V) * 1.2)
    parent = np.array([-1, 0, 0, 0])
    seen = np.zeros(V)
    for _ in range(rounds):
        if kind == "rows":
            x = r.choice(V, 3, p=draft[0].astype(np.float64) / draft[0].astype(np.float64).sum())
        elif kind == "distinct":
            x = np.argsort(-(np.log(draft[0]) + r.gumbel(size=V)))[:3]
        else:
            x = np.argsort(-draft[0])[:3]
        u = r.rand(n).astype(np.float32)
        _, said = tree_plain.verify(target, None if kind == "certain" else draft, [0, *x], parent, u, np.float32(r.rand()), kind == "distinct")
        seen[said[0]] += 1
    want = target[0].astype(np.float64) / target[0].astype(np.float64).sum() * rounds
    assert ((seen - want) ** 2 / want).sum() < 25.7


def test_a_greedy_row_accepts_its_token_alone():
    target = np.zeros((3, 5), dtype=np.float32)
    target[0, 3] = target[1, 1] = target[2, 4] = 1
    for x, path, said in ((3, [0, 1], [3, 1]), (2, [0], [3])):
        for draft in (None, np.full((3, 5), 0.2, dtype=np.float32)):
            got = tree_plain.verify(target, draft, [0, x, 0], [-1, 0, 0], [0.9, 0.99, 0.99], 0.5, False, n=2)
            assert got == (path, said)


# ---- what the library refuses before any launch -------------------------------------------------------------------
P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10002)


def test_tree_attn_refusals(lib):
    s = kvmm.make_shape(1, 1, 4, 1, 64, 16, 64, 8, 64)
    ok = [0, FAKE, 4, None, None, FAKE, FAKE, FAKE, FAKE, None, None, 0.0, FAKE, None, FAKE, 1 << 30, None, None]

    def status(shape=s, **kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.sparse_paged_tree_attn(ctypes.byref(shape), *a)

    for at in (1, 5, 6, 7, 8, 12, 14):  # required arrays
        assert status(**{f"a{at}": None}) == kvmm.INVALID_ARG
        assert status(**{f"a{at}": ODD}) == kvmm.INVALID_ARG
    assert status(a0=1) == kvmm.INVALID_ARG and status(a0=-1) == kvmm.INVALID_ARG
    assert status(a2=0) == kvmm.INVALID_ARG and status(a2=65) == kvmm.UNSUPPORTED_SHAPE
    assert status(a3=ODD) == kvmm.INVALID_ARG  # n_nodes
    assert status(a4=P(0x10004)) == kvmm.INVALID_ARG  # tree_mask: 8-byte words
    assert status(a9=FAKE) == kvmm.INVALID_ARG  # sel_idx without sel_cnt
    assert status(a11=float("nan")) == kvmm.INVALID_ARG and status(a11=3e38) == kvmm.INVALID_ARG
    assert status(a13=ODD) == kvmm.INVALID_ARG and status(a16=ODD) == kvmm.INVALID_ARG
    assert status(a15=8) == kvmm.WORKSPACE_TOO_SMALL
    assert status(kvmm.make_shape(1, 1, 9, 1, 64, 16, 64, 8, 64)) == kvmm.UNSUPPORTED_SHAPE
    assert kvmm.tree_workspace_size(s, 4) > 0
    assert kvmm.tree_workspace_size(s, 0) == 0 and kvmm.tree_workspace_size(s, 65) == 0
    assert kvmm.tree_workspace_size(kvmm.make_shape(1, 1, 4, 1, 96, 16, 64, 8, 64), 4) == 0


def test_draft_verify_refusals(lib):
    ok = [2, 4, 100, FAKE, 100, FAKE, 100, FAKE, FAKE, None, FAKE, FAKE, 0, FAKE, FAKE, FAKE, None, None]

    def status(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.draft_verify(*a)

    for at in (3, 7, 8, 10, 11, 13, 14, 15):
        assert status(**{f"a{at}": None}) == kvmm.INVALID_ARG
        assert status(**{f"a{at}": ODD}) == kvmm.INVALID_ARG
    for at in (5, 9, 16):
        assert status(**{f"a{at}": ODD}) == kvmm.INVALID_ARG
    assert status(a0=0) == kvmm.INVALID_ARG and status(a1=0) == kvmm.INVALID_ARG and status(a2=0) == kvmm.INVALID_ARG
    assert status(a4=99) == kvmm.INVALID_ARG and status(a6=99) == kvmm.INVALID_ARG
    assert status(a12=2) == kvmm.INVALID_ARG
    assert status(a1=65) == kvmm.UNSUPPORTED_SHAPE and status(a0=65536) == kvmm.UNSUPPORTED_SHAPE
    assert status(a4=1 << 41) == kvmm.UNSUPPORTED_SHAPE


def test_keep_path_refusals(lib):
    s = kvmm.make_shape(1, 2, 4, 1, 64, 16, 64, 8, 64)
    ok = [-1, FAKE, FAKE, 4, FAKE, FAKE, FAKE, FAKE, None, None, None]

    def status(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.kv_keep_path(ctypes.byref(s), *a)

    for at in (1, 2, 4, 5, 6, 7):
        assert status(**{f"a{at}": None}) == kvmm.INVALID_ARG
        assert status(**{f"a{at}": ODD}) == kvmm.INVALID_ARG
    assert status(a8=ODD) == kvmm.INVALID_ARG and status(a9=ODD) == kvmm.INVALID_ARG
    assert status(a0=-2) == kvmm.INVALID_ARG and status(a0=2) == kvmm.INVALID_ARG
    assert status(a3=0) == kvmm.INVALID_ARG and status(a3=65) == kvmm.UNSUPPORTED_SHAPE


# ---- what the binding refuses, with tensors that only say that they are on a GPU -------------------------------------
class OnDevice(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def here(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def test_probability_rows_by_their_strides():
    assert kvmm._prob_rows(here(3, 4, 10), "p", 3, 4, 10, 0)[1] == 10
    assert kvmm._prob_rows(here(3, 4, 16)[..., :10], "p", 3, 4, 10, 0)[1] == 16
    assert kvmm._prob_rows(here(1, 4, 16)[..., :10], "p", 1, 4, 10, 0)[1] == 16
    assert kvmm._prob_rows(here(3, 4, 10)[:, :1], "p", 3, 1, 10, 0)[1] == 40  # one node of each tree
    assert kvmm._prob_rows(here(1, 1, 10), "p", 1, 1, 10, 0)[1] == 10


@pytest.mark.parametrize("t", [here(3, 8, 10)[:, ::2], here(3, 4, 20)[..., ::2], here(3, 5, 10)[:, :4],
                               here(3, 10, 4).transpose(1, 2), here(3, 1, 10).expand(3, 4, 10)])
def test_probability_rows_of_other_strides(t):
    if t.stride(1) * t.shape[1] == t.stride(0) and t.stride(2) == 1:  # every other row: evenly spaced after all
        assert kvmm._prob_rows(t, "p", 3, 4, 10, 0)[1] == 20
        return
    with pytest.raises(ValueError, match="p: "):
        kvmm._prob_rows(t, "p", 3, 4, 10, 0)


@pytest.mark.parametrize("t,what", [(here(3, 4, 10, dtype=torch.bfloat16), "float32"), (here(3, 4, 11), "must be"),
                                    (torch.zeros(3, 4, 10), "CUDA")])
def test_probability_rows_refused(t, what):
    with pytest.raises(ValueError, match=what):
        kvmm._prob_rows(t, "p", 3, 4, 10, 0)


def test_node_arrays_are_dense_rows():
    assert kvmm._int_rows(here(2, 3, dtype=torch.int32), "tokens", 2, 3, 0)
    for t in (here(2, 4, dtype=torch.int32), here(6, dtype=torch.int32), here(2, 3, dtype=torch.int64),
              here(2, 6, dtype=torch.int32)[:, ::2], None):
        with pytest.raises(ValueError, match="tokens"):
            kvmm._int_rows(t, "tokens", 2, 3, 0)
