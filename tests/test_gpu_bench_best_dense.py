"""bench.py's speedup against the best dense path: no dense forward of the library that
computes the same is left out of it."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_best_dense_path_counts_both_forwards():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("case bench.py --workload ffn-paper --steps 5 --warmup 1", flush=True)
    r = subprocess.run([sys.executable, "-u", os.path.join(ROOT, "bench.py"), "--workload", "ffn-paper",
                        "--steps", "5", "--warmup", "1", "--no-cpu-baseline", "--no-configs",
                        "--no-fusion-ablation"],
                       cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    d = json.loads([l for l in r.stdout.splitlines() if l.startswith("{")][0])
    times = [d[k]["ms_per_step"] for k in ("dense", "gated_dense", "hipblaslt_dense")]
    assert all(t > 0 for t in times)
    assert abs(d["speedup_vs_best_dense"] - min(times) / d["ms_per_step"]) < 1e-9 * d["speedup_vs_best_dense"]
    assert abs(d["speedup_vs_dense"] - times[0] / d["ms_per_step"]) < 1e-9 * d["speedup_vs_dense"]
    assert abs(d["gated_dense"]["speedup_vs"] - times[1] / d["ms_per_step"]) < 1e-9
