"""Build libdllm.so in place with hipcc for gfx950 (always recompiles)."""
import glob
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(HERE, "libdllm.so")
SOURCES = sorted(glob.glob(os.path.join(HERE, "csrc", "*.hip")))
# Packed-fp32 instructions are turned off for all device code.
FLAGS = ["--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(os.path.dirname(HERE), "include")]
# The step's logits are finite by contract, so NaN handling is compiled out there: max chains map to
# v_max3_f32 without canonicalising each load.  Infinities are still honoured.
FINITE = ["-fno-honor-nans"]
# The calls around the forward take -inf, +inf and NaN and promise what becomes of them, so theirs is
# ordinary arithmetic (at the cost of 16 vector instructions per 4096-column chunk of log probabilities).
NONFINITE_SOURCES = ("logprobs.hip", "embed.hip")


def flags(source):
    """Compiler flags of one source file."""
    return FLAGS if os.path.basename(source) in NONFINITE_SOURCES else FLAGS + FINITE


def _run(cmds, verbose):
    """The commands side by side; CalledProcessError for the first that fails."""
    if verbose:
        for cmd in cmds:
            print(" ".join(cmd), flush=True)
    running = [subprocess.Popen(cmd) for cmd in cmds]
    codes = [p.wait() for p in running]
    for cmd, rc in zip(cmds, codes):
        if rc != 0:
            raise subprocess.CalledProcessError(rc, cmd)


def build(verbose=False, extra=()):
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SOURCES]
        _run([["hipcc", *flags(s), *extra, "-c", "-o", o, s] for s, o in zip(SOURCES, objects)], verbose)
        _run([["hipcc", "--offload-arch=gfx950", "-fPIC", "-shared", "-o", LIB + ".tmp", *objects]], verbose)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
