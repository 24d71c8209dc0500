"""The native part of the binding (_tw_calls.so) shortens the host time of some
calls and is bound to one build of torch: without it the library is still
built, loaded and called.  Nothing here touches a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

PACKAGE = "activation_sparse_feed_gate_amd"


@pytest.fixture(scope="module")
def b():
    """The build module, with both libraries as new as what they are made of."""
    from activation_sparse_feed_gate_amd import build as b

    srcs = [os.path.join(b.CSRC, f) for f in os.listdir(b.CSRC) if f != "peak_probe.hip"]
    srcs.append(os.path.join(b.INCLUDE, "tw.h"))
    newest = max(os.path.getmtime(s) for s in srcs)
    if not all(os.path.exists(p) and os.path.getmtime(p) >= newest for p in (b.LIBRARY, b.CALLS)):
        b.build()
    return b


def imported(root):
    code = (
        "import warnings\n"
        "with warnings.catch_warnings(record=True) as seen:\n"
        "    warnings.simplefilter('always')\n"
        f"    from {PACKAGE} import tw, block\n"
        "print('WARNED', sum('native part' in str(w.message) for w in seen))\n"
        "import torch\n"
        "print('BYTES', tw.tw_workspace_bytes(64, 128, 128, 128, 16, 8) > 0, tw.tw_quant_workspace_bytes(4, 64) > 0)\n"
        "x, g, w = torch.ones(4, 64), torch.ones(64), torch.ones(8, 64, dtype=torch.int8)\n"
        "for f in (lambda: tw.layernorm(x, g), lambda: tw.layernorm_backward(x, x, g, x[:, 0].clone(), x[:, 0].clone()),\n"
        "          lambda: tw.quant_linear(x, w, g[:8]), lambda: tw.quant_gateup(x, w, g[:8], w, g[:8])):\n"
        "    try:\n"
        "        f()\n"
        "    except ValueError as e:\n"
        "        print('REFUSED', 'device tensors' in str(e))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.splitlines()


@pytest.mark.parametrize("calls", ["built", "missing", "unloadable"])
def test_binding_loads_without_the_native_part(b, tmp_path, calls):
    """The sparse FFN and every checked call need libtw.so alone."""
    pkg = tmp_path / PACKAGE
    pkg.mkdir()
    for f in os.listdir(b.HERE):
        if f.endswith(".py") or f in (os.path.basename(b.LIBRARY), os.path.basename(b.CALLS)):
            shutil.copy(os.path.join(b.HERE, f), pkg / f)
    if calls == "missing":
        os.remove(pkg / os.path.basename(b.CALLS))
    elif calls == "unloadable":
        (pkg / os.path.basename(b.CALLS)).write_bytes(b"not a library")
    out = imported(str(tmp_path))
    assert out == [f"WARNED {int(calls != 'built')}", "BYTES True True"] + ["REFUSED True"] * 4


def test_build_keeps_the_library_where_the_native_part_fails(b, tmp_path, monkeypatch):
    """A native part that does not compile fails the build loudly, after the
    library was linked, and leaves no older native part beside it."""
    lib, calls = str(tmp_path / "libtw.so"), tmp_path / "_tw_calls.so"
    calls.write_bytes(b"an older one")
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "LIBRARY", lib)
    monkeypatch.setattr(b, "CALLS", str(calls))
    monkeypatch.setattr(b, "SOURCES", ["tw_api.cpp"])
    monkeypatch.setattr(b, "_calls_flags", lambda: ["-fno-such-flag"])
    with pytest.raises(RuntimeError, match="tw_calls.cpp"):
        b.build()
    assert os.path.exists(lib) and not calls.exists()
