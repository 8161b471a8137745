"""Build step of the ZeRO step library: ``libzero_sm.so`` for sm_100a, and
``_calls.so``, the compiled Python calls.

nvcc cross-compiles without a GPU.  Floating-point flags keep every device
operation IEEE-conformant (no fast-math, no flush to zero, correctly rounded
division and square root, no multiply-add contraction) so that the kernels'
arithmetic is the one stated in ``csrc/kernels.cu``.
"""
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = ["csrc/zero_api.cu", "csrc/kernels.cu", "csrc/fused_tma.cu", "csrc/fused_bulk.cu", "csrc/static_scratch.cu",
           "csrc/two_pass_tma.cu", "csrc/dist.cu", "csrc/guards.cu",
           "csrc/mx4.cu", "csrc/mx4_gemm.cu", "csrc/mx4_gemv.cu", "csrc/mx4_api.cu",
           "csrc/mx8.cu", "csrc/rms_norm.cu", "csrc/embedding.cu", "csrc/layer_api.cu",
           "csrc/plan.cpp"]
LIB = os.path.join(HERE, "libzero_sm.so")
CALLS = os.path.join(HERE, "_calls.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=false",
    "-Xcompiler", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    return shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    from concurrent.futures import ThreadPoolExecutor

    bdir = os.path.join(HERE, "_build")
    os.makedirs(bdir, exist_ok=True)
    cmds, objs = [], []
    for src in SOURCES:
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        cmd = [nvcc(), *NVCC_FLAGS]
        if src.endswith(".cpp"):
            cmd += ["-x", "cu"]
        cmd += ["-c", os.path.join(HERE, src), "-o", obj]
        if ptxas_verbose:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd))
        cmds.append(cmd)
        objs.append(obj)
    # the translation units are independent: compile them side by side
    with ThreadPoolExecutor(max_workers=max(1, min(len(cmds), os.cpu_count() or 1))) as pool:
        for res in pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds):
            if verbose or ptxas_verbose or res.returncode != 0:
                print(res.stdout, end="")
                print(res.stderr, end="")
            if res.returncode != 0:
                raise subprocess.CalledProcessError(res.returncode, res.args, res.stdout, res.stderr)
    # both are made before either is renamed into its place: a reader never sees
    # a half-written file, nor a step that failed half of a new pair
    lib = os.path.join(bdir, os.path.basename(LIB))
    link = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", lib, *objs]
    if verbose:
        print(" ".join(link))
    subprocess.run(link, check=True)
    calls = build_calls(bdir, verbose)
    if calls is None and os.path.exists(CALLS):
        os.remove(CALLS)  # (another library's)
    os.replace(lib, LIB)
    if calls is not None:
        os.replace(calls, CALLS)
    return LIB


def build_calls(bdir: str, verbose: bool = False):
    """``_calls.so`` in ``bdir``: the compiled Python calls, linked to the library
    there and to the torch that is installed.  None where there is none: the
    calls are a shortcut."""
    import importlib.util
    import sysconfig

    torch = importlib.util.find_spec("torch")
    if torch is None or not torch.origin:
        print("torch is not installed: the library is built without its compiled Python calls")
        return None
    torch_dir = os.path.dirname(torch.origin)
    inc = os.path.join(torch_dir, "include")
    out = os.path.join(bdir, os.path.basename(CALLS))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           os.path.join(HERE, "csrc", "calls.cpp"), "-o", out, "-L" + bdir, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    return out


if __name__ == "__main__":
    import sys

    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))
