"""Compile libidx.so (the HIP kernels and the C ABI) for gfx950 with hipcc."""
import glob
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libidx.so")
ARCH = "gfx950"
JOBS = 8

FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 VALU ops are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results go straight to VGPRs: the scoring epilogue reads every
    # accumulator once, so AGPR destinations would cost one v_accvgpr_read each
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall", "-Wno-unused-function",
]


def sources():
    csrc = os.path.join(HERE, "csrc")
    return sorted(glob.glob(os.path.join(csrc, "*.hip"))) + sorted(glob.glob(os.path.join(csrc, "*.cpp")))


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError("libidx build failed:\n" + out)
    return out


def build(verbose: bool = False) -> str:
    """Always recompiles (hipcc cross-compiles gfx950 without a GPU)."""
    tmp = LIB + ".tmp%d" % os.getpid()
    work = tempfile.mkdtemp(prefix="libidx_")
    try:
        def compile_one(src):
            obj = os.path.join(work, os.path.basename(src) + ".o")
            return obj, _run(["hipcc", *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj])

        with ThreadPoolExecutor(JOBS) as pool:
            done = list(pool.map(compile_one, sources()))
        link = _run(["hipcc", "-shared", "-fPIC", f"--offload-arch={ARCH}", *(o for o, _ in done), "-o", tmp])
    finally:
        shutil.rmtree(work, ignore_errors=True)
    out = "\n".join(t for t in [*(t for _, t in done), link] if t.strip())
    if verbose and out.strip():
        print(out)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
