"""The rules by which an int8 product is spread over the chip, on the CPU: the
header that the launchers use, compiled by itself."""
import os
import subprocess

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_rules_over_many_sizes(tmp_path):
    from activation_sparse_feed_gate_amd import build as b

    exe = str(tmp_path / "rules")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-I", b.CSRC, os.path.join(TESTS, "quant_rules_harness.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "RULES_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]
