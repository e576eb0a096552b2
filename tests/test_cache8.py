"""The 8-bit paged cache without a GPU: the model that the GPU tests compare with is checked
against the definitions, and the library and the binding refuse what they must."""
import ctypes

import numpy as np
import pytest
import torch

from tests import cache8_ref as cr


@pytest.fixture(scope="module")
def lib():
    from eviction_gb300 import build
    build.build()
    import eviction_gb300
    return eviction_gb300.load_library()


def test_codes_are_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cr.E4M3_VALUES, want, equal_nan=True)


def test_encoding_is_nearest_even():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(4096, generator=g) * s for s in (1e-3, 0.1, 1, 100)])
    mids = torch.from_numpy(cr._MID).float()
    x = torch.cat([x, mids, -mids, torch.nextafter(mids, torch.tensor(0.0)),
                   torch.nextafter(mids, torch.tensor(500.0))]).clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(cr.encode(x.double().numpy(), cr.E4M3), want)
    y = np.array([0.5, 1.5, -0.5, -2.5, 126.5, 127.4, 300.0, -np.inf, np.nan])
    assert cr.encode(y, cr.INT8).view(np.int8).tolist() == [0, 2, 0, -2, 126, 127, 127, -127, 0]


@pytest.mark.parametrize("fmt,amax,exp", [("e4m3", 448.0, 0), ("e4m3", 450.0, 1), ("e4m3", 224.0, -1),
                                          ("e4m3", 1.0, -8), ("int8", 127.0, 0), ("int8", 127.5, 1),
                                          ("int8", 1.0, -6), ("e4m3", 0.0, -64), ("int8", 3e38, 64),
                                          ("e4m3", 1e-30, -64)])
def test_scale_is_the_smallest_power_of_two(fmt, amax, exp):
    x = np.array([amax / 3, -amax, np.inf, np.nan])
    assert cr.scale_of(x, fmt) == 2.0 ** exp


def test_model_keeps_the_pages_consistent():
    """Random grows, forks and frees: every block is free or counted, none twice."""
    rng = np.random.default_rng(0)
    c = cr.RefCache(1, 8, 1, 8, 40, 4, 12, "int8")
    for _ in range(300):
        what = rng.integers(3)
        if what == 0:
            c.grow(rng.integers(0, 6, 8) * rng.integers(0, 2, 8))
        elif what == 1:
            c.fork(rng.integers(0, 8, 2), rng.permutation(8)[:2])
        else:
            c.free(rng.permutation(8)[:rng.integers(0, 3)])
        held = np.zeros(40, int)
        for b in range(8):
            np.add.at(held, c.table[b, :c.blocks(c.len[b])], 1)
            assert (c.table[b, c.blocks(c.len[b]):] == -1).all()
        assert np.array_equal(held, c.ref)
        free = sorted(c.free_list[:c.top])
        assert free == sorted(np.flatnonzero(held == 0))


def _config(k, **kw):
    return k.Config(**dict(dict(n_layers=2, batch=3, n_kv_heads=2, group=2, head_dim=64, max_T=128,
                                budget=32, window=8), **kw))


def _desc(k, **kw):
    c = k._CCache8(*([4096] * 9), 0, 2, 50, 16, 8)
    for key, val in kw.items():
        setattr(c, key, val)
    return c


@pytest.mark.parametrize("change,code", [
    ({}, 0), (dict(k_pool=0), -1), (dict(ref_count=0), -1), (dict(v_pool=4104), -3),
    (dict(k_scale=4098), -3), (dict(table=4097), -3), (dict(format=2), -1), (dict(format=-1), -1),
    (dict(n_layers=0), -1), (dict(n_blocks=0), -1), (dict(block_size=0), -1),
    (dict(block_size=1025), -1), (dict(block_size=1024), 0), (dict(max_blocks=0), -1),
    (dict(n_blocks=2 ** 31 - 1), -8), (dict(n_blocks=2 ** 26, block_size=16), -8),
    (dict(max_blocks=2 ** 28), -8), (dict(max_blocks=2 ** 29), -8),
    (dict(n_layers=2 ** 30), -8)])
def test_cache_description_is_checked(lib, change, code):
    import eviction_gb300.kvc as k
    cfg = _config(k).c()
    why = ctypes.c_char_p()
    desc = _desc(k, **change)
    assert lib.kvc_cache8_check(ctypes.byref(cfg), ctypes.byref(desc), ctypes.byref(why)) == code
    assert bool(why.value) == (code != 0)
    assert lib.kvc_cache8_check(ctypes.byref(cfg), ctypes.byref(desc), None) == code


def test_null_descriptions(lib):
    import eviction_gb300.kvc as k
    cfg = _config(k).c()
    desc = _desc(k)
    assert lib.kvc_cache8_check(ctypes.byref(cfg), None, None) == -1
    assert lib.kvc_cache8_check(None, ctypes.byref(desc), None) == -1
    bad = _config(k, head_dim=96).c()
    assert lib.kvc_cache8_check(ctypes.byref(bad), ctypes.byref(desc), None) == -8
    d = ctypes.byref(desc)
    assert lib.kvc_cache8_grow(None, d, None, None) == -1
    assert lib.kvc_cache8_append(None, d, None, None, 1, None, None) == -1
    assert lib.kvc_cache8_attend(None, d, None, 1, None, None, None, None) == -1
    assert lib.kvc_cache8_gather(None, d, 1, None, None, None, None) == -1
    assert lib.kvc_cache8_compact(None, d, d, 1, None, None, None, None, None, None) == -1
    assert lib.kvc_cache8_fork(None, d, 1, None, None, None) == -1
    assert lib.kvc_cache8_free(None, d, 1, None, None) == -1


def test_binding_takes_no_cpu_tensors(lib):
    import eviction_gb300 as kvc
    import eviction_gb300.kvc as k
    with pytest.raises(ValueError, match="CUDA"):
        kvc.Cache8.allocate(_config(k), 8, 16, 4, device="cpu")
    with pytest.raises(TypeError, match="float8_e4m3fn or torch.int8"):
        kvc.Cache8.allocate(_config(k), 8, 16, 4, dtype=torch.uint8, device="cpu")
