"""Builds libtk.so (the HIP library behind include/tk.h) for gfx950 with hipcc.

Flags:
  --offload-arch=gfx950           MI355X only
  -ffp-contract=off               no fused multiply-add where the source has two
                                  operations (the ziggurat and the uniform transforms
                                  must round exactly like a plain CPU evaluation)
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                  no packed fp32 instructions
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtk.so")
SOURCES = ["tk_runtime.hip", "tk_fills.hip", "tk_ziggurat.hip", "tk_choice.hip", "tk_rows.hip", "tk_rows_f32.hip",
           "tk_rows_f16.hip", "tk_rows_f16_r32.hip", "tk_rows_bf16.hip", "tk_rows_bf16_r32.hip", "tk_embedding.hip",
           "tk_heads.hip", "tk_checkpoint.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def command(source, out):
    return [
        HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
        "-ffp-contract=off",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall", "-Wno-unused-function",
        "-I", os.path.join(ROOT, "include"), "-I", CSRC,
        "-c", os.path.join(CSRC, source), "-o", out,
    ]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "packed-fp32-ops"  # host pass does not know the device feature
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if ln.strip() and noise not in ln]
    if res.returncode != 0:
        sys.stderr.write("\n".join(msgs) + "\n")
        raise RuntimeError(f"hipcc failed with status {res.returncode}")
    if verbose and msgs:
        print("\n".join(msgs))


def build(verbose: bool = False) -> str:
    """Compiles the sources side by side and links them; the library is replaced at the end."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as d, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        list(pool.map(lambda so: _run(command(*so), verbose), zip(SOURCES, objects)))
        _run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp] + objects, verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
