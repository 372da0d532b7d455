"""The rotated appends and the 4-bit cache at the edges of their formats: values beyond a format's range, infinities,
NaN, signed zeros, and batches that take more than one launch."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import kvmm
from tests import kv4_plain as kp
from tests.test_gpu_append_rope import Case, check_four, fill_pool4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    from paged_kv_cache_minmax_gb300 import build

    build.build_library()
    kvmm.load()
    yield
    torch.cuda.empty_cache()


def append4(c, pool, **kw):
    kvmm.kv4_append_rope(c.shape, c.layer, None, c.k, c.v, c.tb, c.te, pool, c.table, c.meta, rope=c.rope, err=c.err, **kw)
    torch.cuda.synchronize()
    assert int(c.err) == 0


# ---- values beyond the range ----------------------------------------------------------------------------------
@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.5, 1e-38), (1e-38, 0.5), (3.0, 8.0)])
@pytest.mark.parametrize("D,T", [(64, 16), (128, 32)])
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_values_beyond_the_range_saturate(D, T, scales):
    """Infinities, and finite values that leave fp32 times 1 / factor: the scale is 448 and the code +-6."""
    c = Case(Hq=2, D=D, T=T, n=24, begin=(4, 9), end=(28, 33), rope="none", spread=3.0)
    g = np.random.default_rng(11)
    big = float(torch.finfo(torch.bfloat16).max)
    for rows in (c.k, c.v):
        for i in range(24):
            for h in range(2):
                rows[0, i, h, g.integers(D)] = [math.inf, -math.inf, big, -big][i % 4]
                if i % 5 == 0:  # both signs, and next to each other
                    rows[1, i, h, 16:18] = torch.tensor([-math.inf, math.inf])
                    rows[1, i, h, 40] = -big
    pool = fill_pool4(c)
    pool0, meta0 = pool.clone(), c.meta.clone()
    append4(c, pool, k_scale=scales[0], v_scale=scales[1])
    check_four(c, pool0, pool, meta0, *scales)


@pytest.mark.parametrize("rope", ["half", "pairs"])
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_rotations_beyond_the_range_saturate(rope):
    """Pairs whose rotation leaves fp32's range."""
    c = Case(Hq=2, n=24, begin=(4, 9), end=(28, 33), rope=rope)
    big = float(torch.finfo(torch.bfloat16).max)
    c.k.copy_(torch.where(c.k.float().abs() > 1, torch.copysign(torch.full_like(c.k, big), c.k), c.k))
    pool = fill_pool4(c)
    pool0, meta0 = pool.clone(), c.meta.clone()
    append4(c, pool)
    check_four(c, pool0, pool, meta0, 1.0, 1.0)
