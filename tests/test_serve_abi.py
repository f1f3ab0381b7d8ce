"""The entry points of include/qsa_serve.h that need no GPU: exported symbols
and argument checks."""

import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def qsa():
    import __graft_entry__

    __graft_entry__.build()
    from block_sparse_attention_qsa_gb300 import qsa as q

    return q


def test_exports_every_declared_symbol(qsa):
    txt = open(os.path.join(ROOT, "include", "qsa_serve.h")).read()
    code = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    names = set(re.findall(r"\b(qsa_[a-z_0-9]+)\s*\(", code))
    assert names == set(qsa.SERVE_EXPORTS)
    lib = ctypes.CDLL(qsa.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert int(re.search(r"#define QSA_MAX_DRAFTS (\d+)", code).group(1)) == qsa.MAX_DRAFTS
    assert re.search(r"#define QSA_MAX_VOCAB \(1 << 24\)", code) and qsa.MAX_VOCAB == 1 << 24


# made-up device pointers that the calls must refuse before any launch: only
# where no CUDA device exists, so that a regression cannot touch memory
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: CPU-only test")
F = ctypes.c_void_p(1 << 20)
F2 = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 1)
OFF2 = ctypes.c_void_p((1 << 20) + 2)
OFF8 = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40


def _with(args, i, x):
    return [x if k == i else a for k, a in enumerate(args)]


@no_device
def test_prefix_workspace(qsa):
    d = qsa.make_dims(3, 2, 100, 10, 40)
    n, k = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert qsa.lib.qsa_kv_workspace_size(d, ctypes.byref(k)) == qsa.OK
    for pages in (0, 1, 10):
        assert qsa.lib.qsa_prefix_workspace_size(d, pages, ctypes.byref(n)) == qsa.OK
        assert n.value >= k.value and n.value % 256 == 0
    assert qsa.lib.qsa_prefix_workspace_size(d, -1, ctypes.byref(n)) == qsa.ERR_INVALID_ARG
    assert qsa.lib.qsa_prefix_workspace_size(d, 11, ctypes.byref(n)) == qsa.ERR_INVALID_ARG
    assert qsa.lib.qsa_prefix_workspace_size(d, 1, None) == qsa.ERR_INVALID_ARG
    assert qsa.lib.qsa_prefix_workspace_size(None, 1, ctypes.byref(n)) == qsa.ERR_INVALID_ARG
    d.head_dim = 96
    assert qsa.lib.qsa_prefix_workspace_size(d, 1, ctypes.byref(n)) == qsa.ERR_UNSUPPORTED


@no_device
def test_prefix_attn_refusals(qsa):
    d = qsa.make_dims(3, 2, 100, 10, 40, kv_dtype="fp8")
    good = [d, 4, F, F, F, F, F, F, F, F, F, F, F, BIG, None]

    def call(i, x):
        return qsa.lib.qsa_prefix_attn(*_with(good, i, x))

    for i in (2, 3, 4, 5, 6, 7, 8, 9, 10):
        assert call(i, None) == qsa.ERR_INVALID_ARG, i
    assert call(0, None) == qsa.ERR_INVALID_ARG
    for n in (-1, 11):
        assert call(1, n) == qsa.ERR_INVALID_ARG
    for i in (3, 4, 5, 10):
        assert call(i, OFF8) == qsa.ERR_INVALID_ARG, i
    for i in (2, 6, 7, 8, 9, 11):
        assert call(i, OFF2) == qsa.ERR_INVALID_ARG, i
    assert call(12, None) == qsa.ERR_WORKSPACE and call(12, OFF8) == qsa.ERR_WORKSPACE
    assert call(13, 256) == qsa.ERR_WORKSPACE
    n = ctypes.c_size_t(0)
    assert qsa.lib.qsa_prefix_workspace_size(d, 4, ctypes.byref(n)) == qsa.OK
    assert call(13, n.value - 1) == qsa.ERR_WORKSPACE
    for field, val, want in [("head_dim", 96, qsa.ERR_UNSUPPORTED), ("n_q", 5, qsa.ERR_UNSUPPORTED),
                             ("page_size", 48, qsa.ERR_UNSUPPORTED), ("batch", 0, qsa.ERR_INVALID_ARG),
                             ("sm_scale", math.nan, qsa.ERR_INVALID_ARG)]:
        e = qsa.make_dims(3, 2, 100, 10, 40)
        setattr(e, field, val)
        assert call(0, e) == want, field


    for alone in (-1, 2):
        assert qsa.lib.qsa_test_prefix_attn(good[0], alone, *good[1:]) == qsa.ERR_INVALID_ARG
    assert qsa.lib.qsa_test_prefix_attn(good[0], 0, *_with(good, 3, None)[1:]) == qsa.ERR_INVALID_ARG


@no_device
def test_prefix_timeout_hook_refuses_as_prefix_attn(qsa):
    d = qsa.make_dims(3, 2, 100, 10, 40)
    good = [d, 4, F, F, F, F, None, None, F, F, F, F, F, BIG, None]
    for i, x, st in ((0, None, qsa.ERR_INVALID_ARG), (1, 0, qsa.ERR_INVALID_ARG), (1, 11, qsa.ERR_INVALID_ARG),
                     (2, None, qsa.ERR_INVALID_ARG), (10, OFF8, qsa.ERR_INVALID_ARG), (13, 255, qsa.ERR_WORKSPACE)):
        assert qsa.lib.qsa_test_prefix_attn_timeout(*_with(good, i, x)) == st, i


@no_device
def test_kv_weight_refusals(qsa):
    d = qsa.make_dims(3, 2, 100, 10, 40, kv_dtype="fp8")
    good = [d, 0.5, F, F, F, F, F, F, F, F, 256, None]

    def call(i, x):
        return qsa.lib.qsa_kv_weight(*_with(good, i, x))

    for i in (0, 2, 3, 4, 5, 6, 7, 8):
        assert call(i, None) == qsa.ERR_INVALID_ARG, i
    for x in (-0.001, 1.001, math.nan, math.inf):
        assert call(1, x) == qsa.ERR_INVALID_ARG
    for i in (2, 3):
        assert call(i, OFF8) == qsa.ERR_INVALID_ARG
    for i in (4, 5, 6, 7, 8):
        assert call(i, OFF2) == qsa.ERR_INVALID_ARG
    assert call(9, None) == qsa.ERR_WORKSPACE and call(9, OFF8) == qsa.ERR_WORKSPACE and call(10, 255) == qsa.ERR_WORKSPACE
    d.page_size = 8
    assert call(0, d) == qsa.ERR_UNSUPPORTED


@no_device
def test_kv_weight_timeout_hook_refuses_as_kv_weight(qsa):
    d = qsa.make_dims(3, 2, 100, 10, 40)
    good = [d, 0.5, F, F, None, F, F, F, F, F, 256, None]
    for i, x, st in ((0, None, qsa.ERR_INVALID_ARG), (1, 2.0, qsa.ERR_INVALID_ARG), (3, OFF8, qsa.ERR_INVALID_ARG),
                     (7, None, qsa.ERR_INVALID_ARG), (10, 255, qsa.ERR_WORKSPACE)):
        assert qsa.lib.qsa_test_kv_weight_timeout(*_with(good, i, x)) == st, i


@no_device
def test_kv_evict_refusals(qsa):
    d = qsa.make_dims(3, 2, 100, 10, 40)
    #        keep sinks recent out_pages len weight pt  pto kc vc weight_out kept new_len ws
    good = [d, 100, 4, 16, 3, F, F, F, F, F, F, F2, F, F, F, 256, None]

    def call(i, x):
        return qsa.lib.qsa_kv_evict(*_with(good, i, x))

    for i in (0, 5, 6, 7, 8, 9, 10, 11, 12, 13):
        assert call(i, None) == qsa.ERR_INVALID_ARG, i
    for i, x in ((1, 0), (1, -1), (1, 193), (2, -1), (3, -1), (2, 85), (3, 97), (2, 2 ** 31 - 1), (4, 0), (4, -1), (4, 1)):
        assert call(i, x) == qsa.ERR_INVALID_ARG, (i, x)
    for i in (9, 10):
        assert call(i, OFF8) == qsa.ERR_INVALID_ARG
    for i in (5, 6, 7, 8, 11, 12, 13):
        assert call(i, OFF2) == qsa.ERR_INVALID_ARG
    assert call(11, F) == qsa.ERR_INVALID_ARG  # weight_out is weight
    assert call(4, 1 << 25) == qsa.ERR_UNSUPPORTED
    assert call(14, None) == qsa.ERR_WORKSPACE and call(14, OFF8) == qsa.ERR_WORKSPACE and call(15, 255) == qsa.ERR_WORKSPACE


@no_device
def test_verify_drafts_refusals(qsa):
    st = qsa.ProbStrides(400, 100)
    good = [3, 3, 100, 0, F, st, F, None, F, F, F, F, F, 256, None]

    def call(i, x):
        return qsa.lib.qsa_verify_drafts(*_with(good, i, x))

    for i in (4, 8, 9, 10, 11):
        assert call(i, None) == qsa.ERR_INVALID_ARG, i
    for i in (0, 1, 2):
        assert call(i, 0) == qsa.ERR_INVALID_ARG
    for i, x in ((0, (1 << 22) + 1), (1, 32), (2, (1 << 24) + 1), (3, 2), (3, -1)):
        assert call(i, x) == qsa.ERR_UNSUPPORTED, (i, x)
    for i in (4, 6, 8, 9, 10, 11):
        assert call(i, OFF2) == qsa.ERR_INVALID_ARG, i
    assert qsa.lib.qsa_verify_drafts(*_with(_with(good, 3, 1), 6, ODD)) == qsa.ERR_INVALID_ARG
    assert call(12, None) == qsa.ERR_WORKSPACE and call(12, OFF8) == qsa.ERR_WORKSPACE and call(13, 255) == qsa.ERR_WORKSPACE


def test_binding_refuses_host_tensors(qsa):
    d = qsa.make_dims(1, 1, 16, 1, 2)
    i32, f32 = torch.int32, torch.float32
    q = torch.zeros((1, 1, 16, 128), dtype=torch.bfloat16)
    kc = torch.zeros((2, 2, 64, 128), dtype=torch.bfloat16)
    t, one, ws = torch.zeros((1, 1), dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(1024, dtype=torch.uint8)
    w, lse = torch.zeros((1, 64)), torch.zeros((1, 1, 16))
    with pytest.raises(ValueError, match="CUDA"):
        qsa.prefix_attn(d, q, kc, kc, None, None, one, t, t, q, ws)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.kv_weight(d, q, kc, None, t, t, lse, w, ws)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.kv_evict(d, kc, kc, t, t, one, w, w.clone(), t, one, ws)
    p = torch.zeros((1, 2, 10), dtype=f32)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.verify_drafts(p, None, t, torch.zeros((1, 2)), one, torch.zeros((1, 2), dtype=i32), ws)
    with pytest.raises(ValueError, match="target must be"):
        qsa.verify_drafts(p[0], None, t, torch.zeros((1, 2)), one, torch.zeros((1, 2), dtype=i32), ws)
    with pytest.raises(TypeError, match="tensor"):
        qsa.prefix_attn(d, None, kc, kc, None, None, one, t, t, q, ws)


REPORT = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_ZN3qsa1_18prefix_join_kernelILi64ELb0ELi4EEEvNS_10PrefixArgsE' for 'sm_103a'
ptxas info    : Used 77 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN3qsa1_prefix_kernelINS0_2PcILi%dELb%dELi%dEEEEEv14CUtensorMap_st' for 'sm_103a'
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 16 barriers, 1424 bytes smem
"""


def test_build_checks_the_registers_that_warpgroups_share_out():
    from block_sparse_attention_qsa_gb300 import _build

    # (head dim, E4M3, row tiles, registers): 512, 384 and 256 threads
    for good in ((128, 1, 2, 128), (64, 0, 2, 168), (256, 1, 1, 168), (128, 0, 1, 158), (256, 0, 1, 110)):
        assert _build.check_registers(REPORT % good) == 1
    for bad in ((128, 1, 2, 120), (64, 0, 2, 160), (256, 1, 1, 166)):
        with pytest.raises(RuntimeError, match=f"head dim {bad[0]}.*{bad[3]} registers"):
            _build.check_registers(REPORT % (64, 1, 2, 128) + REPORT % bad)
    assert _build.check_registers("ptxas info    : Used 77 registers") == 0


def test_build_stops_at_registers_that_do_not_add_up(monkeypatch, tmp_path):
    from block_sparse_attention_qsa_gb300 import _build

    linked, asked = [], []

    class Done:
        returncode, stdout, stderr = 0, "", REPORT % (128, 1, 2, 120)

    def run(cmd, **kw):
        (linked if "-shared" in cmd else asked).append(cmd)
        return Done()

    for name, to in (("LIB", "lib.so"), ("BUILD", "b")):
        monkeypatch.setattr(_build, name, str(tmp_path / to))
    monkeypatch.setattr(_build, "sources", lambda: [str(tmp_path / "qsa_prefix_128.cu")])
    monkeypatch.setattr(_build, "_newest_input", lambda: 0.0)
    monkeypatch.setattr(_build, "fast_path", lambda: __file__)  # (there already)
    monkeypatch.setattr(_build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="120 registers a thread"):
        _build.build()
    assert len(asked) == 1 and asked[0][asked[0].index("-Xptxas") + 1] == "-v" and not linked
