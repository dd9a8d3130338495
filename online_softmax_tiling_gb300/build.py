"""Build in-tree, without CMake: the sm_103a shared library with nvcc (four translation units)
and, where torch is installed, the torch binding of its paged-cache operators with g++ (one).
The library needs nvcc alone."""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("fa_api.cu", "paged_api.cu", "latent_api.cu", "ceilings.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in ("fa_fwd_kernel.cuh", "fa_fwd_qtile_kernel.cuh", "fa_fwd_wide_kernel.cuh",
                                                     "naive_attention.cuh", "paged_common.cuh", "kv_tables.cuh",
                                                     "kv_append.cuh", "kv_page_select.cuh", "paged_fwd_kernel.cuh",
                                                     "paged_prompt_kernel.cuh", "paged_prompt_wide_kernel.cuh",
                                                     "rotary.cuh", "rotary_host.h", "host_common.h", "latent_append.cuh",
                                                     "latent_paged_kernel.cuh", "latent_fwd_kernel.cuh", "pair_ptx.cuh", "sm103_ptx.cuh")] + [
    os.path.join(ROOT, "include", f) for f in ("fa.h", "fa_ceilings.h", "fa_naive.h", "fa_paged.h", "fa_rotary.h", "fa_latent.h")]
LIBRARY = os.path.join(HERE, "libfa_gb300.so")
BINDING = os.path.join(HERE, "_paged_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_TORCH = BINDING + ".torch"  # the version of torch that BINDING was built for
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
BINDING_DEPENDS = [BINDING_SOURCE, *(os.path.join(ROOT, "include", f) for f in ("fa.h", "fa_paged.h", "fa_rotary.h", "fa_latent.h"))]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise FileNotFoundError("nvcc not found (CUDA 13 toolkit required)")
    return cand


def _stale(target, depends) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in depends)


def _torch_version():
    """The torch's version, None where there is none (imported only if it is not an installed package)."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        pass
    try:
        import torch
        return torch.__version__
    except (ImportError, OSError):
        return None


def _binding_stale() -> bool:
    """Whether there is a torch that the binding does not fit: missing, older than its sources, or built for
    another version (its C++ interface differs from one to the next)."""
    version = _torch_version()
    if version is None:
        return False
    if _stale(BINDING, BINDING_DEPENDS) or not os.path.exists(BINDING_TORCH):
        return True
    with open(BINDING_TORCH, encoding="utf-8") as f:
        return f.read() != version


def stale() -> bool:
    return _stale(LIBRARY, DEPENDS) or _binding_stale()


def _compile_binding(tmp):
    """g++ on the binding: the object only, so that it can run beside nvcc.  None where torch cannot be
    imported: then only callers of the C ABI are served."""
    try:
        from torch.utils.cpp_extension import include_paths
    except (ImportError, OSError) as e:
        print(f"torch cannot be imported ({e}): the torch binding of the paged-cache operators is not built",
              file=sys.stderr)
        return None
    inc = [f"-I{p}" for p in (*include_paths("cuda"), sysconfig.get_paths()["include"])]
    return subprocess.Popen(["g++", "-O2", "-std=c++17", "-fPIC", "-c", "-o", tmp, BINDING_SOURCE, *inc])


def _link_binding(obj):
    """The binding finds the library beside itself, torch's libraries are loaded by `import torch`."""
    from torch.utils.cpp_extension import library_paths
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = [f"-L{p}" for p in library_paths("cuda")] + ["-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch",
                                                        "-lc10_cuda", "-lc10"]
    subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libfa_gb300.so", "-Wl,-rpath,$ORIGIN", *libs],
                   check=True)
    if os.path.exists(BINDING_TORCH):
        os.remove(BINDING_TORCH)
    os.replace(tmp, BINDING)
    with open(BINDING_TORCH, "w", encoding="utf-8") as f:
        f.write(_torch_version() or "")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libfa_gb300.so for sm_103a (static cudart, -O3 -lineinfo) and, where there is a torch, its binding."""
    if not force and not stale():
        return LIBRARY
    obj = BINDING + f".tmp{os.getpid()}.o"
    binding = _compile_binding(obj) if _binding_stale() or (force and _torch_version() is not None) else None
    try:
        if force or _stale(LIBRARY, DEPENDS):
            tmp = LIBRARY + f".tmp{os.getpid()}"
            cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
                   "-Xlinker", "-soname=libfa_gb300.so", "--threads", "4", "-o", tmp, *SOURCES]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            subprocess.run(cmd, check=True)
            os.replace(tmp, LIBRARY)
        if binding is not None:
            if binding.wait() != 0:
                raise subprocess.CalledProcessError(binding.returncode, "g++ torch_binding.cpp")
            _link_binding(obj)
    finally:
        if binding is not None:
            binding.wait()
        if os.path.exists(obj):
            os.remove(obj)
    return LIBRARY


if __name__ == "__main__":
    print(build(force=True, verbose=True))
