"""The products' plan (csrc/fp4q_matmul_plan.h, integer work of the host) as the tests ask for it."""
import collections
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
Plan = collections.namedtuple("Plan", "kernel prepared parts tokens rows waves_k chunk_steps splits split_steps lds workspace refused")


def compiled(folder):
    exe = os.path.join(str(folder), "matmul_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
                    "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "block_scaled_fp4_fp4q_amd", "csrc"),
                    os.path.join(ROOT, "tests", "matmul_plan_driver.cpp"), "-o", exe], check=True)
    return exe


def plans(exe, calls):
    """Of each call (weights, mx, rotate, bf16, rows, cols, tokens)."""
    text = "".join(" ".join(str(int(v)) for v in c) + "\n" for c in calls)
    p = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stderr
    return [Plan(f[0], *(int(v) for v in f[1:])) for f in (line.split() for line in p.stdout.splitlines())]
