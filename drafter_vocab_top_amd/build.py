"""Builds libtopk_cols.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree,
and the compiled part of its Python binding with g++.

    python -m drafter_vocab_top_amd.build

The libraries are placed next to this file; the Python binding loads them from
there.  hipcc cross-compiles for gfx950 without a GPU.  libtopk_cols.so needs
nothing but ROCm: it is in place before the binding is compiled, which is left
out where there is no torch to bind to.
"""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(HERE, "libtopk_cols.so")
SOURCES = [os.path.join(CSRC, n) for n in ("topk_col.hip", "topk_row.hip", "topk_onewave.hip",
                                            "topk_sample.hip", "topk_noalloc.hip", "topk_cols_api.cpp",
                                            "topk_adjust.hip", "topk_count.hip", "topk_verify.hip", "topk_plan.hip",
                                            "topk_round_api.cpp", "topk_tree.hip", "topk_cache.hip", "topk_attend.hip", "topk_attend_rows.hip",
                                            "topk_verify_tree.hip", "topk_cache_api.cpp")]
OBJDIR = os.path.join(ROOT, "_build")
# Per-source flags.  The column kernel takes its ticket before ranking and
# publishing its list and reads the reply afterwards; the compiler's atomic
# optimizer would otherwise wait for the reply right after the atomic (it
# broadcasts the returned value at once), so it is off for that file.  Its
# kernel's leading scalar arguments are preloaded into registers.  The
# row scan asks for three waves per SIMD, which its instantiations with the
# larger candidate area cannot reach; the note saying so is silenced.
EXTRA_FLAGS = {"topk_col.hip": ["-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
                                 "-mllvm", "-amdgpu-kernarg-preload-count=16"],
               "topk_row.hip": ["-Wno-pass-failed"]}
# A plain streaming-read kernel that the benchmark times beside the top-k (not
# part of the top-k library).
STREAM_SOURCE = os.path.join(CSRC, "stream_read.hip")
STREAM_LIBRARY = os.path.join(HERE, "libstream_read.so")
HEADERS = [os.path.join(CSRC, n) for n in ("topk_device.hpp", "topk_col_common.hpp", "topk_internal.hpp", "topk_draw.hpp",
                                            "topk_round.hpp", "topk_lists.hpp", "topk_cache.hpp", "topk_attend.hpp")] + \
          [os.path.join(INCLUDE, "topk_cols.h")]
# The compiled part of the Python binding (host code against torch's headers).
# It holds what it was built for, since it fits no other torch or Python.
BINDING_SOURCE = os.path.join(CSRC, "round_binding.cpp")
BINDING_LIBRARY = os.path.join(HERE, "_round_binding.so")
ARCH = "gfx950"


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def flags():
    return ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
            # keep the compiler from emitting packed fp32 instructions
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-result", "-I", INCLUDE, "-I", CSRC]


def built_for():
    """What the binding's compiled part depends on, torch and Python (None
    without torch)."""
    try:
        import torch
    except ImportError:
        return None
    return f"torch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"


def binding_command(output):
    """The g++ line of the binding's compiled part."""
    import torch
    base = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f'-DTOPK_BUILT_FOR="{built_for()}"',
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-D__HIP_PLATFORM_AMD__", "-I", INCLUDE,
            "-isystem", os.path.join(rocm, "include"), "-isystem", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(base, "include"), "-o", output, BINDING_SOURCE, "-L", os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10"]


def command(output=LIBRARY):
    """One hipcc line that builds the whole library (for reference; the
    per-source flags of EXTRA_FLAGS then apply to every source)."""
    extra = [f for fl in EXTRA_FLAGS.values() for f in fl]
    return [hipcc()] + flags() + extra + ["-shared", "-o", output] + SOURCES


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)


def _check(process, what, verbose):
    _, err = process.communicate()
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in err.splitlines() if noise not in l)
    if process.returncode != 0:
        raise RuntimeError(f"{os.path.basename(process.args[0])} failed on {what} ({process.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build(verbose=False):
    """Compiles every source to an object and the binding in parallel, and
    links the library.  Where the binding fails it raises, with the library in
    place."""
    os.makedirs(OBJDIR, exist_ok=True)
    objs, procs = [], []
    for src in SOURCES + [STREAM_SOURCE]:
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        extra = EXTRA_FLAGS.get(os.path.basename(src), [])
        procs.append((src, _run([hipcc()] + flags() + extra + ["-c", "-o", obj, src], verbose)))
        objs.append(obj)
    binding = _start_binding(verbose)
    for src, process in procs:
        _check(process, os.path.basename(src), verbose)
    for lib, lib_objs in ((LIBRARY, objs[:-1]), (STREAM_LIBRARY, objs[-1:])):
        tmp = lib + ".tmp"
        _check(_run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + lib_objs, verbose), "link", verbose)
        os.replace(tmp, lib)
    bound = False
    try:
        if isinstance(binding, OSError):
            raise RuntimeError(f"the library is built, its Python binding is not: {binding}") from binding
        if binding is not None:
            _check(binding, "the Python binding (the library is built)", verbose)
            os.replace(BINDING_LIBRARY + ".tmp", BINDING_LIBRARY)
            bound = True
    finally:
        # one that was built for the library before this one does not stay
        if not bound and os.path.exists(BINDING_LIBRARY):
            os.remove(BINDING_LIBRARY)
    return LIBRARY


def _start_binding(verbose):
    """The compiler of the binding, the error that kept it from starting, or
    None without a torch to bind to."""
    if built_for() is None:
        print("no torch: the Python binding is left out", file=sys.stderr)
        return None
    try:
        return _run(binding_command(BINDING_LIBRARY + ".tmp"), verbose)
    except OSError as e:
        return e


def stale():
    """Whether a library is missing, older than its sources or, the binding,
    built for another torch or Python."""
    def older(library, sources):
        return not os.path.exists(library) or any(os.path.getmtime(p) > os.path.getmtime(library) for p in sources)
    if older(LIBRARY, SOURCES + HEADERS):
        return True
    this = built_for()
    if this is None:
        return False
    if older(BINDING_LIBRARY, [BINDING_SOURCE] + HEADERS):
        return True
    with open(BINDING_LIBRARY, "rb") as f:
        return this.encode() + b"\0" not in f.read()


if __name__ == "__main__":
    print(build(verbose=True))
