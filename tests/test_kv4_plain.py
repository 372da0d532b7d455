"""The plain 4-bit and rotation arithmetic of tests/kv4_plain.py against torch and brute force, and the refusals of
the entry points that use it (host side only)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_minmax_gb300 import build, kvmm
from tests import kv4_plain as kp


def test_e4m3_matches_torch():
    x = np.concatenate([np.linspace(0, 448, 20011), kp.E4M3, (kp.E4M3[1:] + kp.E4M3[:-1]) / 2,
                        np.exp2(np.linspace(-14, 8.8, 5000))]).astype(np.float32)
    want = torch.from_numpy(x).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kp.nearest(x.astype(np.float64), kp.E4M3).astype(np.uint8), want)


def test_e2m1_nearest_is_nearest_with_ties_to_even():
    x = np.linspace(0, 8, 6401)
    got = kp.LEVELS[kp.nearest(x, kp.LEVELS)]
    d = np.abs(x[:, None] - kp.LEVELS)
    assert np.array_equal(np.abs(x - got), d.min(1))
    for tie, level in ((0.25, 0), (0.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (3.5, 4), (5.0, 4), (7.0, 6)):
        assert kp.LEVELS[kp.nearest(np.array([tie]), kp.LEVELS)][0] == level


def test_held_values_are_exact_in_bf16_and_close():
    rng = np.random.default_rng(0)
    x = kp.bf16(rng.standard_normal((200, 64)) * np.exp2(rng.integers(-12, 12, (200, 1))))
    for scale in (1.0, 0.37, 4.0):
        codes, s = kp.hold(x, scale)
        v = kp.value(codes, s)
        assert np.array_equal(kp.bf16(v), v)
        g = np.abs(kp.f32(x * np.float64(np.float32(1) / np.float32(scale)))).reshape(200, 4, 16)
        # half the widest step of e2m1 (1 of 6) plus the scale's own rounding (2^-4, or half a subnormal step)
        lim = g.max(-1) * (1 / 6 + 2.0 ** -4) + 6 * 2.0 ** -10
        live = g.max(-1) < 2600
        err = np.abs(v.reshape(200, 4, 16) - (x / scale).reshape(200, 4, 16)).max(-1)
        assert (err <= lim * 1.0001)[live].all()


def test_rotation_keeps_lengths_and_distance_dependence():
    rng = np.random.default_rng(1)
    D, dim = 64, 64
    inv = 10000.0 ** (-2.0 * np.arange(dim // 2) / dim)
    q, k = rng.standard_normal(D), rng.standard_normal(D)
    for inter in (False, True):
        turn = lambda x, t: kp.rotate(x, np.cos(t * inv), np.sin(t * inv), dim, inter, rounded=False)  # noqa: E731
        assert abs(np.linalg.norm(turn(q, 17)) - np.linalg.norm(q)) < 1e-12
        assert abs(turn(q, 25) @ turn(k, 20) - turn(q, 105) @ turn(k, 100)) < 1e-10


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return kvmm.load()


S = kvmm.make_shape(2, 1, 4, 2, 64, 16, 8, 4, 64)


def test_sizes(lib):
    assert kvmm.kv4_page_bytes(S) == 16 * (32 + 4) * 2
    assert kvmm.kv4_page_bytes(kvmm.make_shape(1, 1, 4, 1, 128, 32, 8, 4, 8)) == 32 * 72 * 2
    assert kvmm.kv4_page_bytes(kvmm.make_shape(1, 1, 4, 1, 96, 16, 8, 4, 8)) == 0
    assert kvmm.kv4_workspace_size(S) > 0
    assert kvmm.kv4_workspace_size(kvmm.make_shape(1, 1, 36, 4, 64, 16, 8, 4, 8)) == 0


def _rows(**kw):
    a = dict(data=0x10000, batch_stride=1024, token_stride=512, head_stride=64)
    a.update(kw)
    return ctypes.byref(kvmm.Rows(a["data"], a["batch_stride"], a["token_stride"], a["head_stride"]))


def _rope(**kw):
    a = dict(table=0x20000, positions=None, rows=100, dim=64, interleaved=0)
    a.update(kw)
    return ctypes.byref(kvmm.RopeStruct(a["table"], a["positions"], a["rows"], a["dim"], a["interleaved"]))


def _append(lib, four, shape=S, layer=0, q=None, k=None, v=None, n=1, tb=0x30000, te=0x30000, rope=None, q_out=None,
            pool=0x40000, table=0x50000, meta=0x60000, scale=1.0, err=None):
    k, v = k or _rows(), v or _rows()
    if four:
        return lib.kv4_append_rope(ctypes.byref(shape), layer, q, k, v, n, tb, te, rope, q_out, pool, scale, scale,
                                   table, meta, err, None)
    return lib.kv_append_rope(ctypes.byref(shape), layer, q, k, v, n, tb, te, rope, q_out, pool, pool, table, meta,
                              err, None)


BAD_APPEND = {
    "layer": dict(layer=1), "no rows": dict(n=0), "negative rows": dict(n=-3),
    "misaligned rows": dict(k=_rows(data=0x10008)), "no data": dict(v=_rows(data=None)),
    "odd stride": dict(k=_rows(token_stride=100)), "negative stride": dict(v=_rows(head_stride=-64)),
    "q without q_out": dict(q=_rows()), "q_out without q": dict(q_out=0x70000),
    "misaligned q_out": dict(q=_rows(), q_out=0x70004), "no begin": dict(tb=None), "no end": dict(te=None),
    "misaligned pool": dict(pool=0x40008), "no pool": dict(pool=None), "no table": dict(table=None),
    "misaligned meta": dict(meta=0x60002), "misaligned err": dict(err=0x70002),
    "rope without table": dict(rope=_rope(table=None)), "misaligned rope": dict(rope=_rope(table=0x20004)),
    "rope of no rows": dict(rope=_rope(rows=0)), "rope wider than a row": dict(rope=_rope(dim=96)),
    "rope of nothing": dict(rope=_rope(dim=0)), "rope pairing": dict(rope=_rope(interleaved=2)),
    "misaligned positions": dict(rope=_rope(positions=0x30002)),
}


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("name", sorted(BAD_APPEND))
def test_append_refuses(lib, name, four):
    assert _append(lib, four, **BAD_APPEND[name]) == kvmm.INVALID_ARG


@pytest.mark.parametrize("four", [False, True])
def test_append_refuses_shapes(lib, four):
    assert _append(lib, four, rope=_rope(dim=16)) == kvmm.UNSUPPORTED_SHAPE
    assert _append(lib, four, shape=kvmm.make_shape(1, 1, 4, 2, 80, 16, 8, 4, 64)) == kvmm.UNSUPPORTED_SHAPE
    assert _append(lib, four, shape=kvmm.make_shape(1, 1, 5, 2, 64, 16, 8, 4, 64)) == kvmm.INVALID_ARG


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf"), 1e-39])
def test_factors_are_refused(lib, scale):
    assert _append(lib, True, scale=scale) == kvmm.INVALID_ARG
    f = 0x10000
    assert lib.kv4_gather(ctypes.byref(S), 0, f, scale, 1.0, f, None, f, 4, f, f, None, None) == kvmm.INVALID_ARG
    assert lib.sparse_paged_decode_attn_kv4(ctypes.byref(S), 0, f, f, 1.0, scale, f, f, None, None, 0.0, f, None, f,
                                            1 << 24, 0, None, None) == kvmm.INVALID_ARG


def test_gather_refuses(lib):
    f = 0x10000
    ok = [0, f, 1.0, 1.0, f, None, f, 4, f, f, None, None]
    for at, bad in ((0, -1), (0, 1), (1, None), (1, f + 8), (4, None), (5, f + 2), (6, None), (7, 0), (8, f + 2),
                    (9, f + 8), (10, f + 1)):
        a = list(ok)
        a[at] = bad
        assert lib.kv4_gather(ctypes.byref(S), *a) == kvmm.INVALID_ARG, (at, bad)
    a = list(ok)
    a[8] = a[9] = None
    assert lib.kv4_gather(ctypes.byref(S), *a) == kvmm.INVALID_ARG


def test_attention_refuses(lib):
    f = 0x10000
    ok = [0, f, f, 1.0, 1.0, f, f, f, f, 0.0, f, None, f, 1 << 24, 0, None, None]
    for at, bad in ((0, 1), (1, None), (1, f + 8), (2, None), (2, f + 4), (5, None), (6, None), (7, None), (8, None),
                    (7, f + 2), (9, float("nan")), (9, float("inf")), (9, 3e38), (10, None), (10, f + 2), (11, f + 1),
                    (12, None), (12, f + 8), (14, 2), (15, f + 2)):
        a = list(ok)
        a[at] = bad
        assert lib.sparse_paged_decode_attn_kv4(ctypes.byref(S), *a) == kvmm.INVALID_ARG, (at, bad)
    a = list(ok)
    a[13] = kvmm.kv4_workspace_size(S) - 1
    assert lib.sparse_paged_decode_attn_kv4(ctypes.byref(S), *a) == kvmm.WORKSPACE_TOO_SMALL
    a = list(ok)
    assert lib.sparse_paged_decode_attn_kv4(ctypes.byref(kvmm.make_shape(1, 1, 9, 1, 64, 16, 8, 4, 64)),
                                            *a) == kvmm.UNSUPPORTED_SHAPE


def test_binding_refuses_cpu_tensors_and_shapes():
    t = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kvmm._rows(t, "new_k", 2, 1, 2, 64, 0)
    with pytest.raises(ValueError, match="dim|table"):
        kvmm.Rope(torch.zeros(4, 2, 16), 64)
    with pytest.raises(ValueError, match="CUDA"):
        kvmm.Rope(torch.zeros(4, 2, 32), 64)
    with pytest.raises(ValueError, match="together"):
        kvmm.sparse_paged_decode_attn_kv4(S, 0, t, t, t, t, t, None, t, t)
    with pytest.raises(ValueError, match="required"):
        kvmm.kv4_gather(S, 0, t, t, None, t, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        kvmm._arg(t, "q", torch.bfloat16, 1, 0)
    with pytest.raises(ValueError, match="required"):
        kvmm._arg(None, "q", torch.bfloat16, 1, 0)
