"""The paged cache's entry points refuse bad arguments on the host (no GPU
needed), and the 64-bit reference of the GPU tests holds to its definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_band_b200 as pb
from tests import cache_ref as R

A = 1 << 20  # an address that no call here gets to use


def _cfg(**kw):
    args = dict(requests=3, page=64, num_pages=40, max_pages=9, hq=8, hkv=2, tokens=12, max_add=4)
    args.update(kw)
    return pb.PrismCacheConfig(**args)


def _calls(cfg, ws=1 << 40):
    return {
        "plan": pb.lib.prism_cache_plan(cfg.ptr(), *[A] * 9, None),
        "store": pb.lib.prism_cache_store(cfg.ptr(), A, 0, 0, A, 0, 0, *[A] * 5, None),
        "attn": pb.lib.prism_cache_attn(cfg.ptr(), A, 0, 0, *[A] * 7, None, A, A, ws, None),
        "size": pb.lib.prism_cache_workspace_size(cfg.ptr(), ctypes.byref(ctypes.c_size_t())),
    }


@pytest.mark.parametrize("kw,code", [
    (dict(requests=0), -2), (dict(requests=4097), -6), (dict(page=0), -6), (dict(page=48), -6), (dict(page=256), -6),
    (dict(num_pages=0), -2), (dict(max_pages=-1), -2), (dict(hq=7), -2), (dict(hkv=0), -2), (dict(hq=130, hkv=2), -6),
    (dict(head_dim=64), -6), (dict(tokens=0), -2), (dict(max_add=0), -2), (dict(max_add=13), -2),
    (dict(num_pages=1 << 25), -2), (dict(max_pages=1 << 25), -2),
    (dict(page_stride=2 * 64 * 128 - 16), -2), (dict(page_stride=2 * 64 * 128 + 8), -3), (dict(page_stride=1 << 40), -6),
])
def test_bad_config_refused(kw, code):
    for name, s in _calls(_cfg(**kw)).items():
        assert s == code, (name, s)


def test_null_and_unaligned_arguments_refused():
    c = _cfg()
    for i in range(9):
        for bad, code in ((None, -1), (A + 2, -3)):
            args = [A] * 9
            args[i] = bad
            assert pb.lib.prism_cache_plan(c.ptr(), *args, None) == code, i
    # store: k, v, slots, k_cache, v_cache, k_scale, v_scale
    for i, align in enumerate((8, 8, 2, 8, 8, 2, 2)):
        for bad, code in ((None, -1), (A + align, -3)):
            a = [A] * 7
            a[i] = bad
            assert pb.lib.prism_cache_store(c.ptr(), a[0], 0, 0, a[1], 0, 0, *a[2:], None) == code, i
    for strides in ((4, 128), (256, 4), (12, 0)):
        assert pb.lib.prism_cache_store(c.ptr(), A, *strides, A, 0, 0, *[A] * 5, None) == -3
        assert pb.lib.prism_cache_attn(c.ptr(), A, *strides, *[A] * 7, None, A, A, 1 << 40, None) == -3
    assert pb.lib.prism_cache_store(c.ptr(), A, 0, 0, A, -256, 128, *[A] * 5, None) == -2
    # attn: q, k_cache, v_cache, k_scale, v_scale, table, lens, starts, mask, o
    for i, align in enumerate((8, 8, 8, 2, 2, 2, 2, 2, 2, 8)):
        for bad, code in ((None, -1), (A + align, -3)):
            if i == 8 and bad is None:
                continue  # no mask
            a = [A] * 10
            a[i] = bad
            assert pb.lib.prism_cache_attn(c.ptr(), a[0], 0, 0, *a[1:], A, 1 << 40, None) == code, i
    need = pb.prism_cache_workspace_size(c)
    assert need > 0 and need % 256 == 0
    assert pb.lib.prism_cache_attn(c.ptr(), A, 0, 0, *[A] * 8, A, A, need - 1, None) == -7
    assert pb.lib.prism_cache_attn(c.ptr(), A, 0, 0, *[A] * 8, A, None, need, None) == -7
    assert pb.lib.prism_cache_attn(c.ptr(), A, 0, 0, *[A] * 8, A, A + 16, need, None) == -3
    assert pb.lib.prism_cache_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == -1
    assert pb.lib.prism_cache_workspace_size(c.ptr(), None) == -1


def test_binding_refuses_wrong_tensors():
    c = _cfg()
    host = torch.zeros(12, 2, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(4000, dtype=torch.int32)
    with pytest.raises(ValueError):
        pb.prism_cache_store(c, host, host, A, A, A, A, A, stream=0)
    with pytest.raises(ValueError):  # too few entries, wrong type
        pb.prism_cache_plan(c, i32[:2], A, A, A, A, A, A, A, stream=0)
    with pytest.raises(ValueError):
        pb.prism_cache_plan(c, i32.long(), A, A, A, A, A, A, A, stream=0)
    with pytest.raises(ValueError):
        pb.prism_cache_attn(c, A, A, A, A, A, A, A, A, host, None, stream=0)


def test_error_code_has_a_description():
    assert "cache" in pb.prism_status_str(-13)
    assert _cfg(max_pages=65, page=64).words == 2 and _cfg(max_pages=64, page=64).words == 1


def test_reference_codes_agree_with_torch():
    """The reference's table and rounding are e4m3's: every code, every midpoint, their neighbours."""
    codes = torch.arange(256, dtype=torch.uint8)
    theirs = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.E4M3, theirs, equal_nan=True)
    mag = R.E4M3[:127]
    x = np.concatenate([mag, (mag[1:] + mag[:-1]) / 2, np.nextafter(np.float32((mag[1:] + mag[:-1]) / 2), np.float32(0))])
    x = np.concatenate([x, -x]).astype(np.float32)
    assert np.array_equal(R.encode(x), torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("amax", [448.0, 449.0, 447.0, 1.75, 1.7578125, 3.5, 2.0 ** -100, 3.3e38, 0.0])
def test_reference_scale_is_the_smallest_power_of_two(amax):
    s = R.page_scale(np.array([amax, -amax / 2, math.nan, math.inf]))
    assert math.frexp(s)[0] == 0.5 and amax / s <= 448.0
    assert s == 2.0 ** -64 or 2 * amax / s > 448.0


def test_reference_plan_conserves_pages():
    """Steps of growing, idle and ending requests: no page is in two places, none is lost."""
    rng = np.random.default_rng(3)
    n, page, num, wide = 6, 16, 60, 12
    ring, state, table = rng.permutation(num).astype(np.int32), np.array([17, num, 0, 0]), np.full((n, wide), -1)
    held = np.zeros(n, np.int64)
    for step in range(60):
        add = np.where(rng.random(n) < 0.15, -1, rng.integers(0, 40, n))
        add = np.where(held + add > wide * page, -1, add)
        lens, starts, slots, ring, state, table = R.plan(held, add, ring, state, table, page, 300)
        free = [ring[(state[0] + k) % num] for k in range(state[1])]
        used = [table[i, j] for i in range(n) for j in range(-(-lens[i] // page))]
        assert sorted(free + used) == list(range(num))
        live = slots[slots >= 0]
        assert len(set(live.tolist())) == len(live) == starts[-1]
        held = lens.astype(np.int64)


@pytest.fixture
def builder(monkeypatch, tmp_path):
    """build.py with its outputs in an empty folder and the compilers' runs recorded instead of made."""
    import importlib.util
    import os
    import types
    path = os.path.join(os.path.dirname(pb.__file__), "build.py")
    spec = importlib.util.spec_from_file_location("_prism_build_test", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(mod, "BIND", str(tmp_path / "bind.so"))
    mod.fails = ""

    def run(cmd, **kw):
        if mod.fails and mod.fails in cmd[0]:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(mod, "subprocess", types.SimpleNamespace(run=run))
    return mod


def test_library_is_built_where_the_binding_cannot_be(builder, monkeypatch):
    import os
    import sys
    builder.fails = "g++"
    with pytest.raises(RuntimeError):
        builder.build()
    assert os.path.exists(builder.LIB) and not os.path.exists(builder.BIND)
    os.remove(builder.LIB)
    builder.fails = ""
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)  # (import torch raises ImportError)
        assert builder.build() == builder.LIB
    assert os.path.exists(builder.LIB) and not os.path.exists(builder.BIND)
    builder.build()
    assert os.path.exists(builder.BIND)


@pytest.mark.parametrize("lens,adds,group,hkv", [([300, 128], [128, 128], 2, 2), ([365, 65], [65, 65], 1, 1), ([5, 2], [5, 2], 64, 1),
                                                 ([6000, 700, 300], [150, 40, 300], 4, 2), ([500, 77], [130, 50], 2, 3)])
def test_crowded_calls_of_the_gpu_tests_run_the_tile_kernel(lens, adds, group, hkv):
    from tests.test_gpu_cache_kernels import crowded, takes_tiles
    assert not takes_tiles(lens, adds, group, hkv, max(adds))
    assert takes_tiles(*crowded(lens, adds, group, hkv), group, hkv, 200)
