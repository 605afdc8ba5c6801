"""The work decomposition of the prompt-weights kernel, enumerated on the CPU
(tests/c/weights_plan_check.cu): every pair of query and key once in each pass."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_pair_is_computed_once_in_each_pass(tmp_path):
    exe = str(tmp_path / "weights_plan_check")
    subprocess.run(["nvcc", "-O2", "-std=c++17", "-o", exe, os.path.join(ROOT, "tests", "c", "weights_plan_check.cu")],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout
