"""The few-token kernel's weight stream (csrc/few_stream.h) on the host: with every wait in turn running out, no stage is
loaded before its chunk was taken, and no copy is on its way when the block leaves."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sparse_moe_layer_joint_b200", "csrc")


def test_stream_keeps_its_rules_when_a_wait_runs_out(tmp_path):
    exe = str(tmp_path / "few_stream_check")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, os.path.join(HERE, "few_stream_check.cpp"),
                           "-o", exe])
    done = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0 and done.stdout.startswith("ok "), done.stdout
    assert int(done.stdout.split()[1]) > 1000
