"""Host tests of the serving calls (dg_kv_append, dg_paged_attention, dg_adjust_logits) at the edge of what
include/dg.h allows; nothing is launched."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import entropy_bounded_denoising_gb300 as dg
from entropy_bounded_denoising_gb300 import _native, build


def _kv(**kw):
    f = dict(k=16, v=16, page_table=16, kv_len=16, n_pages=4, page_stride=16 * 128, slot_stride=128,
             head_stride=128, page_size=16, max_pages=4)
    f.update(kw)
    return _native._PagedKV(*(f[n] for n, _ in _native._PagedKV._fields_))


def _attention(q=16, o=32, lse=None, cu=16, causal=16, n=1, mq=4, total=4, Hq=2, Hkv=1, D=128, W=-1, scale=0.1, ws=256,
               wsb=None, kv=None):
    need = dg.dg_paged_attention_workspace_bytes(n, mq, Hq, Hkv, D)
    c = _kv() if kv is None else kv
    return dg.load().dg_paged_attention(q, ctypes.byref(c), o, lse, cu, causal, n, mq, total, Hq, Hkv, D, W, scale, ws,
                                        need if wsb is None else wsb, None)


def test_scales_whose_log2_form_is_infinite_are_refused():
    for scale in (3e38, -3e38, 1.8e38, float("nan"), float("inf")):
        assert _attention(scale=scale) == dg.DG_ERR_INVALID_ARG
    for scale in (2.0 ** 127, -2.0 ** 127, 0.0):   # past this check: the workspace's is next
        assert _attention(scale=scale, ws=None) == dg.DG_ERR_WORKSPACE


def _append(k=16, ldk=128, v=16, ldv=128, q=16, ldq=256, qo=32, cu=16, n=1, total=4, Hq=2, Hkv=1, D=128, w=16, rot=128,
            kv=None):
    c = _kv() if kv is None else kv
    return dg.load().dg_kv_append(k, ldk, v, ldv, q, ldq, qo, cu, n, total, Hq, Hkv, D, w, rot, 0, ctypes.byref(c), None)


def _adjust(x=16, dt=0, ld=64, out=32, ldo=64, n=1, L=4, V=64, p=16, h=16, cuh=16, nh=5, pen=16, bt=16, bv=16, cub=16,
            nb=5, m=16, ms=2, nm=1, mi=16):
    return dg.load().dg_adjust_logits(x, dt, ld, out, ldo, n, L, V, p, h, cuh, nh, pen, bt, bv, cub, nb, m, ms, nm, mi,
                                      None)


def test_pointers_between_their_elements_are_refused():
    """A kernel's read of a word that does not lie on a multiple of its size ends the context; records given as
    bytes, and pointers through the C ABI, may lie anywhere."""
    for off in (1, 2, 3):
        for name in ("p", "h", "cuh", "pen", "bt", "bv", "cub", "m", "mi"):
            assert _adjust(**{name: 16 + off}) == dg.DG_ERR_ALIGNMENT, name
        for kw in (dict(cu=16 + off), dict(lse=16 + off), dict(kv=_kv(page_table=16 + off)), dict(kv=_kv(kv_len=16 + off))):
            assert _attention(**kw) == dg.DG_ERR_ALIGNMENT, kw
        for kw in (dict(cu=16 + off), dict(w=16 + 4), dict(w=16 + off), dict(kv=_kv(page_table=16 + off)),
                   dict(kv=_kv(kv_len=16 + off))):
            assert _append(**kw) == dg.DG_ERR_ALIGNMENT, kw


def test_the_workspace_for_a_larger_call_serves_the_smaller_ones():
    """With the same heads the size never falls as the sequences or their queries grow."""
    counts = [1, 2, 3, 8, 17, 64, 150, 256, 1000, 65535]
    queries = [1, 2, 3, 4, 5, 8, 9, 16, 17, 64, 128, 129, 256, 300, 2048, 1 << 20]
    for D in (64, 128, 256):
        for Hq, Hkv in ((1, 1), (8, 8), (16, 8), (32, 4), (40, 1), (71, 1)):
            size = {(n, q): dg.dg_paged_attention_workspace_bytes(n, q, Hq, Hkv, D) for n in counts for q in queries}
            for i, n in enumerate(counts):
                for j, q in enumerate(queries):
                    assert size[n, q] > 0
                    assert i == 0 or size[n, q] >= size[counts[i - 1], q], (n, q, Hq, Hkv, D)
                    assert j == 0 or size[n, q] >= size[n, queries[j - 1]], (n, q, Hq, Hkv, D)


def test_the_step_needs_the_library_alone():
    """Without the serving calls' Python module the library loads and the other calls work; a serving call says what
    is missing."""
    code = ("import entropy_bounded_denoising_gb300 as dg, torch\n"
            "from entropy_bounded_denoising_gb300 import _native\n"
            "_native._build.BIND = '/nonexistent/dg_bind.so'\n"
            "lib = dg.load()\n"
            "assert dg.dg_denoise_workspace_bytes(1, 16, 1024) > 0 and dg.version() >= 100\n"
            "assert lib.dg_denoise_step(None, 0, 8, 1, 16, 8, None, 0, *([None] * 11), None, 0, None) == dg.DG_ERR_INVALID_ARG\n"
            "assert dg.dg_paged_attention_workspace_bytes(1, 1, 8, 8, 64) > 0\n"
            "x = torch.zeros((1, 4, 64))\n"
            "try:\n"
            "    dg.dg_adjust_logits(x, torch.zeros(36, dtype=torch.uint8))\n"
            "except RuntimeError as e:\n"
            "    assert 'build_bind' in str(e)\n"
            "else:\n"
            "    raise AssertionError('no error')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("how", ["no compiler", "no headers"])
def test_the_library_builds_without_what_the_python_module_needs(monkeypatch, tmp_path, how):
    build.build()
    run, old = subprocess.run, tmp_path / "dg_bind.so"
    old.write_bytes(b"of another source")
    os.utime(old, (0, 0))

    def fails(cmd, **kw):
        if cmd[0] != "g++":
            return run(cmd, **kw)
        if how == "no compiler":
            raise FileNotFoundError("g++")
        return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")

    monkeypatch.setattr(build, "BIND", str(old))
    monkeypatch.setattr(build.subprocess, "run", fails)
    with pytest.warns(UserWarning, match="serving calls"):
        assert build.build() == build.LIB
    assert not old.exists()              # a stale one is not left to be loaded
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build_bind()


@pytest.mark.parametrize("shape,order,alike", [((3, 8, 1, 64), (0, 2, 1, 3), True), ((1, 8, 2, 64), (1, 0, 2, 3), True),
                                               ((1, 8, 1, 64), (2, 1, 0, 3), True), ((3, 8, 2, 64), (0, 2, 1, 3), False)])
def test_strides_of_extents_of_one_may_differ(shape, order, alike):
    """The stride of an extent of one says nothing: caches that differ in it alone have one layout."""
    k = torch.zeros(shape, dtype=torch.bfloat16)
    v = torch.zeros([shape[i] for i in order], dtype=torch.bfloat16).permute(order)
    assert v.shape == k.shape and v.stride() != k.stride()
    x = torch.zeros((4, shape[2], 64), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="device tensors" if alike else "one layout"):   # the check that comes next
        dg.dg_kv_append(x, x, k, v, i32(1, 3), i32(2), i32(1))
