"""Builds libssu.so (the gfx950 kernels and the C-ABI entry points) in-tree
with hipcc, and the layer operators' Python module over it with g++."""
import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssu.so")
SOURCES = [os.path.join(CSRC, "ssu_kernels.hip"), os.path.join(CSRC, "ssu_replay.hip"),
           os.path.join(CSRC, "ssu_copy.hip"),
           os.path.join(CSRC, "ssu_ssd.hip"), os.path.join(CSRC, "ssu_noalloc.hip"),
           os.path.join(CSRC, "ssu_norm.hip"), os.path.join(CSRC, "ssu_mx.hip"),
           os.path.join(CSRC, "ssu_logprob.hip"),
           os.path.join(CSRC, "ssu_api.cpp"), os.path.join(CSRC, "ssu_layer_api.cpp")]
# Streaming-ceiling kernels for the benchmark (a separate library, not part
# of libssu's interface).
CEILING_SRC = os.path.join(CSRC, "ssu_ceiling.hip")
CEILING_LIB = os.path.join(HERE, "libssu_ceiling.so")
# The layer operators' Python functions (torch tensors in and out), linked
# against libssu.so beside them.
TORCH_SRC = os.path.join(CSRC, "ssu_torch.cpp")
TORCH_LIB = os.path.join(HERE, "_ssu_torch.so")
HEADERS = [os.path.join(CSRC, "ssu_internal.h"), os.path.join(CSRC, "ssu_device.h"),
           os.path.join(CSRC, "ssu_layer.h"), os.path.join(CSRC, "ssu_layer_device.h"),
           os.path.join(os.path.dirname(HERE), "include", "ssu.h")]

# Packed-fp32 instructions are switched off for all device code; hipcc -O3
# still vectorises loads, stores and conversions.
HIPCC_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-fvisibility=hidden"]


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def torch_command(obj):
    """g++ command that compiles TORCH_SRC to `obj`, and the libraries to link it with."""
    import torch
    root = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(rocm, "include")]
    flags = ["-O2", "-D__HIP_PLATFORM_AMD__", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    libs = ["-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10",
            "-L" + os.path.join(rocm, "lib"), "-lamdhip64"]
    return ["g++", *flags, *["-I" + i for i in inc], "-c", "-o", obj, TORCH_SRC], libs


def build(out=LIB, extra=(), ceiling=True):
    """Compile the library into `out` (always recompiles), and the ceiling
    library next to the package; returns `out`. The package's own library
    comes with the Python module over it.

    Each source is compiled to its own object in parallel (no relocatable
    device code: every translation unit carries its own kernels), then the
    objects are linked."""
    tag = "%s.%d" % (os.path.basename(out), os.getpid())
    srcs = SOURCES + ([CEILING_SRC] if ceiling else [])
    objs = [os.path.join(os.path.dirname(out), "_%s_%s.o" % (os.path.basename(src), tag))
            for src in srcs]

    torch_obj = os.path.join(os.path.dirname(out), "_%s_%s.o" % (os.path.basename(TORCH_SRC), tag))
    module = out == LIB
    torch_compile, torch_libs = torch_command(torch_obj) if module else (None, None)

    def compile_one(i):
        cmd = torch_compile
        if i < len(srcs):
            cmd = [hipcc(), *HIPCC_FLAGS, *extra, "-c", "-o", objs[i], srcs[i]]
        subprocess.run(cmd, check=True)

    def link(lib, parts, command=(hipcc(), "--offload-arch=gfx950")):
        tmp = lib + ".tmp%d" % os.getpid()
        subprocess.run([*command, "-shared", "-fPIC", "-o", tmp, *parts], check=True)
        os.replace(tmp, lib)

    try:
        jobs = max(1, min(len(srcs), int(os.environ.get("MAX_JOBS", "4"))))
        with ThreadPoolExecutor(jobs) as pool:
            list(pool.map(compile_one, range(len(srcs) + module)))
        link(out, objs[:len(SOURCES)])
        if module:
            # by its bare name: a path would be looked up as it is, past the rpath
            link(TORCH_LIB, [torch_obj, *torch_libs, "-L" + os.path.dirname(out),
                             "-l:" + os.path.basename(out), "-Wl,-rpath,$ORIGIN"], ["g++"])
        if ceiling:
            link(CEILING_LIB, objs[len(SOURCES):])
    finally:
        for o in objs + [torch_obj]:
            if os.path.exists(o):
                os.remove(o)
    return out


def stale(lib=LIB):
    if not os.path.exists(lib) or (lib == LIB and not os.path.exists(TORCH_LIB)):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in SOURCES + HEADERS + [TORCH_SRC])


if __name__ == "__main__":
    print(build())
