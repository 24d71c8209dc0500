"""The host checks of the layer-norm and int8 entry points under
AddressSanitizer and UndefinedBehaviorSanitizer (host side only), driven by
norm_quant_host_harness.cpp through the extremes of every size.  Nothing
touches a GPU."""
import os
import subprocess

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_host_validation_under_asan_ubsan(tmp_path):
    from activation_sparse_feed_gate_amd import build as b

    kernels = [os.path.join(b.BUILD_DIR, s + ".o") for s in b.SOURCES if s.endswith(".hip")]
    if not all(os.path.exists(o) for o in kernels):
        b.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host",
           "-fno-omit-frame-pointer"]
    flags = [x for x in b.FLAGS if x != "-fPIC"] + ["-g"]
    objs = []
    for src in (os.path.join(b.CSRC, "tw_api.cpp"), os.path.join(TESTS, "norm_quant_host_harness.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run([b.HIPCC, *flags, *san, "-x", "hip", "-c", src, "-o", obj], check=True,
                       capture_output=True)
        objs.append(obj)
    exe = str(tmp_path / "harness")
    subprocess.run([b.HIPCC, "--offload-arch=gfx950", *san, *objs, *kernels, "-o", exe],
                   check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "HARNESS_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
    assert "runtime error" not in r.stderr, r.stderr[-3000:]
