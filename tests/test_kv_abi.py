"""The entry points of include/qsa_kv.h that need no GPU: exported symbols,
the rotary frequency table against its formulas, and argument checks."""

import ctypes
import math
import os
import re
import subprocess
import sys
import sysconfig

import numpy as np
import pytest
import torch

from tests import _kv_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def qsa():
    import __graft_entry__

    __graft_entry__.build()
    from block_sparse_attention_qsa_gb300 import qsa as q

    return q


def test_exports_every_declared_symbol(qsa):
    txt = open(os.path.join(ROOT, "include", "qsa_kv.h")).read()
    m = re.search(r"#define QSA_MAX_KV_HEADS (\d+)", txt)
    assert m and int(m.group(1)) == qsa.MAX_KV_HEADS
    names = set(re.findall(r"\b(qsa_[a-z_0-9]+)\s*\(", re.sub(r"/\*.*?\*/", "", txt, flags=re.S)))
    assert names == set(qsa.KV_EXPORTS)
    lib = ctypes.CDLL(qsa.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("rot_dim", [2, 4, 6, 64, 128, 256])
@pytest.mark.parametrize("kw", [
    dict(), dict(base=5e5), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
    dict(scaling="yarn", factor=40.0, orig_len=4096.0), dict(scaling="yarn", factor=1.0, orig_len=1.0),
    dict(scaling="yarn", factor=8.0, orig_len=8192.0, alpha=1.0, beta=4.0),
], ids=str)
def test_rope_table_is_the_formula(qsa, rot_dim, kw):
    if kw.get("scaling") == "ntk" and rot_dim == 2:
        with pytest.raises(qsa.QSAError):  # the exponent rot_dim / (rot_dim - 2) has no value
            qsa.rope_table(rot_dim, **kw)
        return
    turns, amp = qsa.rope_table(rot_dim, **kw)
    w, want_amp = R.frequencies(rot_dim, **kw)
    # pow, divisions and the constant pi in 64 bits: relative 2^-53 each, a
    # handful of them (NTK's base passes through pow twice, whose exponent
    # magnifies the error of the base by at most 1), then half of 2^-64
    assert np.all(np.abs(turns.astype(np.float64) * 2.0 ** -64 - w / (2 * math.pi)) <= 2.0 ** -49 * w + 2.0 ** -64)
    assert abs(amp - want_amp) <= 2.0 ** -24 * want_amp


def test_rope_table_amplitude_given(qsa):
    assert qsa.rope_table(64, amplitude=0.75)[1] == 0.75
    assert qsa.rope_table(64, scaling="yarn", factor=4.0, orig_len=100.0, amplitude=2.0)[1] == 2.0


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=-2), dict(rot_dim=8, base=1.0),
    dict(rot_dim=8, base=float("nan")), dict(rot_dim=8, base=float("inf")),
    dict(rot_dim=8, scaling="linear", factor=0.5), dict(rot_dim=8, scaling="linear", factor=float("nan")),
    dict(rot_dim=8, scaling="yarn", factor=2.0), dict(rot_dim=8, scaling="yarn", factor=2.0, orig_len=float("inf")),
    dict(rot_dim=8, scaling="yarn", factor=2.0, orig_len=10.0, alpha=4.0, beta=4.0),
    dict(rot_dim=8, scaling="yarn", factor=2.0, orig_len=10.0, alpha=-1.0, beta=4.0),
    dict(rot_dim=8, amplitude=-1.0), dict(rot_dim=8, amplitude=float("nan")), dict(rot_dim=8, amplitude=1e300),
    dict(rot_dim=4, scaling="ntk", factor=1e300),
], ids=str)
def test_rope_table_refusals(qsa, kw):
    with pytest.raises(qsa.QSAError) as e:
        qsa.rope_table(**kw)
    assert e.value.status == qsa.ERR_INVALID_ARG


def test_rope_table_refuses_unknown_enumerators_and_nulls(qsa):
    turns, amp = np.zeros(64, np.uint64), ctypes.c_float(0)
    for layout, scaling in ((2, 0), (-1, 0), (0, 4), (0, -1)):
        spec = qsa.RopeSpec(8, layout, scaling)
        assert qsa.lib.qsa_rope_table(spec, turns.ctypes.data, amp) == qsa.ERR_INVALID_ARG
    ok = qsa.RopeSpec(8, 0, 0)
    assert qsa.lib.qsa_rope_table(ok, None, amp) == qsa.ERR_INVALID_ARG
    assert qsa.lib.qsa_rope_table(None, turns.ctypes.data, amp) == qsa.ERR_INVALID_ARG
    assert qsa.lib.qsa_rope_table(ok, turns.ctypes.data, None) == qsa.ERR_INVALID_ARG


# made-up device pointers that the calls must refuse before any launch: only
# where no CUDA device exists, so that a regression cannot touch memory
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: CPU-only test")
F = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
OFF8 = ctypes.c_void_p((1 << 20) + 8)


def _size(qsa, d):
    n = ctypes.c_size_t(0)
    return qsa.lib.qsa_kv_workspace_size(ctypes.byref(d), ctypes.byref(n)), n.value


@no_device
def test_geometry(qsa):
    for D in (64, 128, 256):
        for hq, hk in ((16, 2), (1, 1), (12, 4), (7, 1), (1024, 8)):
            st, n = _size(qsa, qsa.make_dims(3, 2, 100, 10, 40, n_q_heads=hq, n_kv_heads=hk, head_dim=D))
            assert st == qsa.OK and n >= 256
    for field, val, want in [("head_dim", 96, "U"), ("n_q", 5, "U"), ("page_size", 48, "U"), ("page_size", 8, "U"),
                             ("page_size", 512, "U"), ("n_q_heads", 17, "U"), ("n_q_heads", 1026, "U"),
                             ("kv_dtype", 7, "U"), ("max_pages", 1 << 26, "U"), ("batch", 0, "I"), ("n_q", 0, "I"),
                             ("num_pages", 0, "I"), ("max_pages", -1, "I"), ("n_kv_heads", 0, "I"),
                             ("sm_scale", float("nan"), "I"), ("sm_scale", -1.0, "I"), ("sm_scale", float("inf"), "I")]:
        d = qsa.make_dims(1, 4, 100, 10, 10)
        setattr(d, field, val)
        want = qsa.ERR_UNSUPPORTED if want == "U" else qsa.ERR_INVALID_ARG
        assert _size(qsa, d)[0] == want, field
        assert qsa.lib.qsa_paged_attn(d, 0, F, F, F, None, None, F, F, F, None, F, 1 << 40, None) == want, field
        assert qsa.lib.qsa_kv_gather(d, 1, F, F, None, None, F, F, F, F, F, 256, None) == want, field
        assert qsa.lib.qsa_kv_append(d, 1, None, F, None, F, None, None, None, None, None, F, F, F, F, None, None, F,
                                     256, None) == want, field
    assert qsa.lib.qsa_kv_workspace_size(None, None) == qsa.ERR_INVALID_ARG


@no_device
def test_paged_attn_refusals(qsa):
    d = qsa.make_dims(2, 4, 100, 10, 10)
    n = _size(qsa, d)[1]
    good = [d, 0, F, F, F, None, None, F, F, F, F, F, n, None]
    call = qsa.lib.qsa_paged_attn
    for i in (2, 3, 4, 7, 8, 9):  # q, caches, page table, positions, out
        assert call(*[None if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, i
    for i in (2, 3, 4, 9):  # 16-byte alignment
        assert call(*[OFF8 if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, i
    for i in (7, 8, 10):
        assert call(*[ODD if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, i
    assert call(*[-1 if k == 1 else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG
    assert call(*[n - 1 if k == 12 else a for k, a in enumerate(good)]) == qsa.ERR_WORKSPACE
    assert call(*[OFF8 if k == 11 else a for k, a in enumerate(good)]) == qsa.ERR_WORKSPACE
    assert call(*[None if k == 11 else a for k, a in enumerate(good)]) == qsa.ERR_WORKSPACE
    d8 = qsa.make_dims(2, 4, 100, 10, 10, kv_dtype="fp8")
    assert call(d8, 0, F, F, F, None, F, F, F, F, None, F, 1 << 40, None) == qsa.ERR_INVALID_ARG


@no_device
def test_append_and_gather_refusals(qsa):
    d = qsa.make_dims(2, 1, 100, 10, 10)
    rope = qsa.RopeArgs(128, 0, 1.0, 1 << 20)
    good = [d, 5, rope, F, None, F, None, F, None, F, None, F, F, F, F, None, None, F, 256, None]
    call = qsa.lib.qsa_kv_append
    for i in (3, 5, 11, 12, 13, 14):
        assert call(*[None if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, i
    for i in (3, 5, 7, 9, 11, 12):
        assert call(*[ODD if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, i
    for i in (13, 14):
        assert call(*[OFF8 if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, i
    for i, bad in ((1, 0), (1, -1), (1, qsa.MAX_CHUNK + 1), (2, None), (7, None), (9, None)):
        assert call(*[bad if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, (i, bad)
    for bad in (qsa.RopeArgs(130, 0, 1.0, 1 << 20), qsa.RopeArgs(0, 0, 1.0, 1 << 20), qsa.RopeArgs(5, 0, 1.0, 1 << 20),
                qsa.RopeArgs(64, 2, 1.0, 1 << 20), qsa.RopeArgs(64, 0, 0.0, 1 << 20),
                qsa.RopeArgs(64, 0, math.nan, 1 << 20), qsa.RopeArgs(64, 0, 1.0, None),
                qsa.RopeArgs(64, 0, 1.0, (1 << 20) + 4)):
        assert call(*[bad if k == 2 else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG
        assert qsa.lib.qsa_rope(bad, 1, 1, 1, 128, 0, F, None, F, F, None, None) == qsa.ERR_INVALID_ARG
    # an output whose elements coincide, and an output over its input in another order
    assert call(*[qsa.Strides(0, 2048, 128) if k == 10 else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG
    assert call(*[qsa.Strides(1 << 20, 4096, 128) if k == 8 else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG
    for ws, n in ((None, 256), (OFF8, 256), (F, 255)):
        assert call(*(good[:17] + [ws, n, None])) == qsa.ERR_WORKSPACE
        assert qsa.lib.qsa_kv_gather(d, 5, F, F, None, None, F, F, F, F, ws, n, None) == qsa.ERR_WORKSPACE
    d8 = qsa.make_dims(2, 1, 100, 10, 10, kv_dtype="fp8")
    assert call(*([d8] + good[1:])) == qsa.ERR_INVALID_ARG
    g = [d, 5, F, F, None, None, F, F, F, F, F, 256, None]
    for i in (2, 3, 6, 7, 8, 9):
        assert qsa.lib.qsa_kv_gather(*[None if k == i else a for k, a in enumerate(g)]) == qsa.ERR_INVALID_ARG, i
    for i in (2, 3, 8, 9):
        assert qsa.lib.qsa_kv_gather(*[OFF8 if k == i else a for k, a in enumerate(g)]) == qsa.ERR_INVALID_ARG, i
    assert qsa.lib.qsa_kv_gather(*([d8] + g[1:])) == qsa.ERR_INVALID_ARG


@no_device
def test_rope_refusals(qsa):
    rope = qsa.RopeArgs(64, 0, 1.0, 1 << 20)
    call = qsa.lib.qsa_rope
    good = [rope, 2, 3, 4, 64, 0, F, None, F, F, None, None]
    for i in (0, 6, 8, 9):
        assert call(*[None if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, i
    for i, bad in ((1, 0), (2, 0), (3, 0), (5, 2), (5, -1), (6, ODD), (8, ODD), (9, ODD)):
        assert call(*[bad if k == i else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG, (i, bad)
    for i, bad in ((4, 32), (4, 96), (3, 1025)):
        assert call(*[bad if k == i else a for k, a in enumerate(good)]) == qsa.ERR_UNSUPPORTED, (i, bad)
    assert call(rope, 1 << 16, 1 << 15, 1, 64, 0, F, None, F, F, None, None) == qsa.ERR_UNSUPPORTED
    for st in (qsa.Strides(0, 256, 64), qsa.Strides(768, 0, 64), qsa.Strides(768, 256, 0)):
        assert call(*[st if k == 10 else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG
    # in place only with the same strides
    assert call(*[qsa.Strides(2000, 256, 64) if k == 7 else a for k, a in enumerate(good)]) == qsa.ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_bad_arguments(qsa):
    bf, i32 = torch.bfloat16, torch.int32
    d = qsa.make_dims(1, 1, 16, 1, 1)
    x = torch.zeros(1, 1, 16, 128, dtype=bf)
    kv = torch.zeros(1, 1, 2, 128, dtype=bf)
    cache = torch.zeros(1, 2, 64, 128, dtype=bf)
    pos, ws = torch.zeros(1, 1, dtype=i32), torch.zeros(4096, dtype=torch.uint8)
    rope = qsa.make_rope(128, device="cpu")
    with pytest.raises(ValueError, match="CUDA|current device"):
        qsa.rope(rope, x, pos, x)
    with pytest.raises(TypeError, match="make_rope"):
        qsa.rope(None, x, pos, x)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.kv_append(d, kv, kv, cache, cache, None, None, pos, pos, ws)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.kv_gather(d, cache, cache, None, None, pos, pos, kv, kv, ws)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.paged_attn(d, x, cache, cache, None, None, pos, pos, x, ws)
    with pytest.raises(ValueError, match="window"):
        qsa.paged_attn(d, x, cache, cache, None, None, pos, pos, x, ws, window=1 << 32)
    with pytest.raises(KeyError):
        qsa.make_rope(128, layout="other", device="cpu")


# --------------------------------------------------------------------------
# the binding's fast path
# --------------------------------------------------------------------------
def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_fast_path_is_built_for_this_python_and_torch(qsa):
    from block_sparse_attention_qsa_gb300 import _build

    path = _build.fast_path()
    assert os.path.exists(path) and qsa._fast.__file__ == path
    assert torch.__version__ in path and path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_build_makes_a_missing_fast_path_and_nothing_else(qsa, monkeypatch, tmp_path):
    # (after a change of Python or torch: the library is newer than every source)
    from block_sparse_attention_qsa_gb300 import _build

    monkeypatch.setattr(_build, "fast_path", lambda: str(tmp_path / "_fast.other.so"))
    before = os.path.getmtime(_build.LIB)
    assert _build.build() == _build.LIB
    assert (tmp_path / "_fast.other.so").exists() and os.path.getmtime(_build.LIB) == before
    made = os.path.getmtime(tmp_path / "_fast.other.so")
    _build.build()
    assert os.path.getmtime(tmp_path / "_fast.other.so") == made


def test_build_goes_on_without_a_fast_path(qsa, monkeypatch, tmp_path):
    from block_sparse_attention_qsa_gb300 import _build

    monkeypatch.setattr(_build, "fast_path", lambda: str(tmp_path / "_fast.other.so"))
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    with pytest.warns(RuntimeWarning, match="not built"):
        assert _build.build() == _build.LIB


@pytest.mark.parametrize("stale", [False, True])
def test_binding_works_without_its_fast_path(qsa, stale, tmp_path):
    # missing, or a file that this Python cannot load: the library is all that
    # the binding needs, and a call gets the same checks
    path = tmp_path / "_fast.other.so"
    if stale:
        path.write_bytes(b"built for something else")
    r = _python(f"""
import warnings
from block_sparse_attention_qsa_gb300 import _build
_build.fast_path = lambda: {str(path)!r}
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    from block_sparse_attention_qsa_gb300 import qsa
assert any("fast path is not there" in str(x.message) for x in w), w
assert qsa.rope_table(64)[1] == 1.0 and qsa.workspace_size(qsa.make_dims(1, 1, 16, 1, 1)) > 0
import torch
t = torch.zeros((1, 1, 2, 128), dtype=torch.bfloat16)
try:
    qsa.rope(qsa.make_rope(64, device="cpu"), t, torch.zeros((1, 1), dtype=torch.int32), t)
except ValueError as e:
    assert "cuda" in str(e).lower(), e
else:
    raise AssertionError("a host tensor was taken")
print("fine")
""")
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
