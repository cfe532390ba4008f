"""Build libw4a16.so in-tree with nvcc for sm_103a (no GPU needed to compile), and the
Python module of the serving step's calls, which links it, with the host compiler."""
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libw4a16.so")
MODULE = os.path.join(OUT_DIR, "_w4a16_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    for cand in (shutil.which("nvcc"), os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_header():
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(h) for h in hdrs)


def _module_commands(obj, out):
    """To compile csrc/binding.cpp against the installed torch, and to link it with libw4a16.so."""
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] +
                   ["-I" + i for i in inc] + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])
    link_cmd = ["g++", "-shared", obj, "-o", out, "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                "-L" + OUT_DIR, "-lw4a16", "-Wl,-rpath," + lib, "-Wl,-rpath,$ORIGIN"]
    return compile_cmd, link_cmd


def build(force=False, verbose=False, ptxas_verbose=False):
    """Compile each csrc/*.cu and the Python module in parallel, then link libw4a16.so. Returns the library path."""
    os.makedirs(os.path.join(OUT_DIR, "obj"), exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = _newest_header()
    objs, procs = [], []
    for src in srcs:
        obj = os.path.join(OUT_DIR, "obj", os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        stale = force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time)
        if stale:
            cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    binding, module_obj = os.path.join(CSRC, "binding.cpp"), os.path.join(OUT_DIR, "obj", "binding.o")
    module_stale = (force or not os.path.exists(module_obj) or
                    os.path.getmtime(module_obj) < max(os.path.getmtime(binding), hdr_time))
    if module_stale:
        cmd, _ = _module_commands(module_obj, None)
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        module = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    logs = []
    for src, pr in procs:
        out, _ = pr.communicate()
        logs.append(out.decode(errors="replace"))
        if pr.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s" % (src, logs[-1]))
    if procs or force or not os.path.exists(LIB):
        tmp = LIB + ".tmp%d" % os.getpid()
        subprocess.check_call([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    if module_stale:
        out, _ = module.communicate()
        logs.append(out.decode(errors="replace"))
        if module.returncode != 0:
            raise RuntimeError("g++ failed on %s:\n%s" % (binding, logs[-1]))
    if module_stale or not os.path.exists(MODULE):
        tmp = MODULE + ".tmp%d" % os.getpid()
        subprocess.check_call(_module_commands(module_obj, tmp)[1])
        os.replace(tmp, MODULE)
    if verbose or ptxas_verbose:
        sys.stderr.write("".join(logs))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
