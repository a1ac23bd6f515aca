"""Host-side edges of the head's operators (no GPU needed)."""
import ctypes
import importlib.machinery
import importlib.metadata
import os
import random
import subprocess

import pytest

torch = pytest.importorskip("torch")
from test_layers_host import BF16, E4M3, F32, INV, OK, lib  # noqa: F401,E402


def _ptrs(values):
    return (ctypes.c_void_p * len(values))(*values)


def _adamw(lib, p, g, m, v, sizes, ms=None, vs=None, c=None):
    return lib.uf_adamw_step(len(p), _ptrs(p), _ptrs(g), _ptrs(m), _ptrs(v), ms and _ptrs(ms), vs and _ptrs(vs), c and _ptrs(c),
                             (ctypes.c_int64 * len(p))(*sizes), F32, BF16, E4M3 if ms else F32, 1e-3, None, 0.9, 0.999, 1e-8,
                             0.01, 1, None, 0, None, None)


def test_adamw_refuses_overlaps_across_tensors(lib):
    """Any two of 40 tensors' 240 buffers made to share their last and first byte, in lists of rising,
    falling and random addresses.  (Device addresses that are never followed; every call is refused.)"""
    rng = random.Random(1)
    n, page = 40, 1 << 20
    for order in ("up", "down", "random"):
        slots = list(range(1, 6 * n + n + 1))
        if order == "down":
            slots.reverse()
        elif order == "random":
            rng.shuffle(slots)
        lists = [[page * s for s in slots[i * n:(i + 1) * n]] for i in range(7)]
        sizes = [rng.choice((1, 255, 256, 257, 1000)) for _ in range(n)]
        p, m, v, ms, vs, c, g = range(7)
        elem = {p: 4, m: 1, v: 1, ms: 4, vs: 4, c: 2, g: 2}

        def extent(which, i):
            return elem[which] * (-(-sizes[i] // 256) if which in (ms, vs) else sizes[i])

        for _ in range(200):
            a, b = rng.randrange(7), rng.randrange(6)  # b is written
            i, j = rng.sample(range(n), 2)
            moved = [list(x) for x in lists]
            # a's buffer ends on b's first element, or starts on its last one
            if rng.random() < 0.5:
                end = (moved[b][j] + elem[b] + 3) // 4 * 4
                moved[a][i] = end - (extent(a, i) + 3) // 4 * 4
            else:
                moved[a][i] = (moved[b][j] + extent(b, j) - elem[b]) // 4 * 4
            lo, hi = max(moved[a][i], moved[b][j]), min(moved[a][i] + extent(a, i), moved[b][j] + extent(b, j))
            if lo >= hi:
                continue
            args = [moved[k] for k in (p, g, m, v)]
            assert _adamw(lib, *args, sizes, moved[ms], moved[vs], moved[c]) == INV, (order, a, i, b, j)


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """build.py on an empty folder, with compilers that only write their output file; the list of their calls."""
    from contrastive_embedding_loss_gb300 import build

    calls = []

    def run(cmd, **kw):
        calls.append(os.path.basename(cmd[0]))
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    return build, calls, monkeypatch


def test_the_library_builds_without_torch(compilers):
    build, calls, monkeypatch = compilers

    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    monkeypatch.setattr(build.importlib.metadata, "version", missing)
    out = build.build()
    assert os.path.exists(out) and not os.path.exists(build.native_path())
    assert calls == ["nvcc"] * (len(build.SOURCES) + 1)


def test_the_library_builds_beside_a_torch_without_cuda(compilers, tmp_path):
    build, calls, monkeypatch = compilers
    spec = importlib.machinery.ModuleSpec("torch", None, origin=str(tmp_path / "torch" / "__init__.py"))
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)
    out = build.build()
    assert os.path.exists(out) and not os.path.exists(build.native_path()) and "g++" not in calls


def test_another_torch_rebuilds_the_binding_alone(compilers):
    build, calls, monkeypatch = compilers
    build.build()
    assert sorted(calls) == ["g++"] + ["nvcc"] * (len(build.SOURCES) + 1) and os.path.exists(build.native_path())
    calls.clear()
    build.build()
    assert calls == []
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0.1")
    build.build()
    assert calls == ["g++"]


def test_a_binding_of_another_torch_is_not_loaded(lib, monkeypatch):
    from contrastive_embedding_loss_gb300 import layers

    assert layers._load_native() is not None
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1" if name == "torch" else version(name))
    with pytest.raises(ImportError, match="not built for this torch"):
        layers._load_native()
