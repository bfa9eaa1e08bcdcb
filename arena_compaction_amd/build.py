"""Build libarena_compaction.so (gfx950) in-tree with hipcc."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_PATH = os.path.join(HERE, "libarena_compaction.so")
SOURCES = ["api.cpp", "monitor.cpp", "readback.cpp", "plan.hip", "move.hip", "remap.hip",
           "publish.hip", "static.hip", "kv_api.cpp", "kv_append.hip", "kv_attend.hip",
           "kv_prompt.hip", "kv_finish.hip", "kv_evict.hip"]
ARCH = "gfx950"  # MI355X (CDNA4) only

# No packed-FP32 instructions anywhere in the device code.  hipcc hands the
# feature to the host pass as well, where x86 does not know it and says so
# once per function ("... is not a recognized feature for this target
# (ignoring feature)"); clang cannot forward an option that takes an argument
# to the device pass alone, so that one harmless line is dropped from the
# compiler's output below and everything else is shown.
NO_PACKED_FP32 = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
HOST_FEATURE_NOTE = "'-packed-fp32-ops' is not a recognized feature for this target (ignoring feature)"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wextra",
    *NO_PACKED_FP32,
    "-I", os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    return os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def run_hipcc(cmd) -> None:
    """Run a hipcc command; show its output except the host pass's note
    about the device-only feature; raise on failure."""
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    shown = [ln for ln in p.stdout.splitlines() if ln.strip() != HOST_FEATURE_NOTE]
    if shown:
        print("\n".join(shown), file=sys.stderr, flush=True)
    if p.returncode != 0:
        raise subprocess.CalledProcessError(p.returncode, cmd)


def build(verbose: bool = False, extra_flags=()) -> str:
    """Each source to an object, several at a time, then one link."""
    flags = [hipcc()] + HIPCC_FLAGS + list(extra_flags)
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, s + ".o") for s in SOURCES]
        compiles = [[f for f in flags if f != "-shared"] + ["-c", os.path.join(CSRC, s), "-o", o]
                    for s, o in zip(SOURCES, objects)]
        link = [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared"] + objects + ["-o", LIB_PATH + ".tmp"]
        if verbose:
            for cmd in compiles + [link]:
                print(" ".join(cmd), flush=True)
        jobs = min(8, os.cpu_count() or 1, int(os.environ.get("MAX_JOBS") or 8))
        with concurrent.futures.ThreadPoolExecutor(max(1, jobs)) as pool:
            list(pool.map(run_hipcc, compiles))
        run_hipcc(link)
    os.replace(LIB_PATH + ".tmp", LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
