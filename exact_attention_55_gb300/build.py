"""Build the CUDA library in-tree: exact_attention_55_gb300/_build/libgb300attn.so.

Every translation unit is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``), in parallel, then linked into
one shared library with the CUDA runtime linked statically.  The kernel file
``attn_fwd_inst.cu`` is compiled once per (head dim, operand type) pair.  Beside it,
``csrc/binding.cpp`` becomes a Python extension against the installed PyTorch
(``_build/_gb300attn_binding.so``): host code only, compiled by the host compiler.  What it
was built against (PyTorch and Python versions) is kept in a file beside it; another one makes it stale.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB_NAME = "libgb300attn.so"
LIB_PATH = os.path.join(BUILD, LIB_NAME)
BINDING_NAME = "_gb300attn_binding"
BINDING_PATH = os.path.join(BUILD, BINDING_NAME + ".so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + CSRC, "-I" + INCLUDE]

# (object name, source, extra defines)
UNITS = [
    ("api", "api.cu", []),
    ("quant_fp8", "quant_fp8.cu", []),
    ("decode", "decode.cu", []),
    ("decode_tc", "decode_tc.cu", []),
    ("decode_fp8_wide", "decode_fp8_wide.cu", []),
    ("decode_fp8", "decode_fp8.cu", []),
    ("paged", "paged.cu", []),
    ("attn_bwd", "attn_bwd.cu", []),
    ("fwd_bf16_d64", "attn_fwd_inst.cu", ["-DGB300_ATTN_D=64", "-DGB300_ATTN_F8=0"]),
    ("fwd_bf16_d128", "attn_fwd_inst.cu", ["-DGB300_ATTN_D=128", "-DGB300_ATTN_F8=0"]),
    ("fwd_bf16_d256", "attn_fwd_inst.cu", ["-DGB300_ATTN_D=256", "-DGB300_ATTN_F8=0"]),
    ("fwd_fp8_d64", "attn_fwd_inst.cu", ["-DGB300_ATTN_D=64", "-DGB300_ATTN_F8=1"]),
    ("fwd_fp8_d128", "attn_fwd_inst.cu", ["-DGB300_ATTN_D=128", "-DGB300_ATTN_F8=1"]),
    ("fwd_fp8_d256", "attn_fwd_inst.cu", ["-DGB300_ATTN_D=256", "-DGB300_ATTN_F8=1"]),
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths.append(os.path.join(INCLUDE, "attn.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _abi() -> str:
    """What the binding's binary interface depends on."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _binding_abi_path() -> str:
    return BINDING_PATH + ".abi"


def _binding_abi() -> str:
    """What the binding on disk was built against ("" if unknown)."""
    try:
        with open(_binding_abi_path(), encoding="utf-8") as f:
            return f.read()
    except OSError:
        return ""


def _compile_binding() -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *("-I" + i for i in inc),
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stderr}")
    # the versions last: a run that ends in between leaves a binding that counts as stale
    with contextlib.suppress(FileNotFoundError):
        os.remove(_binding_abi_path())
    os.replace(tmp, BINDING_PATH)
    with open(tmp, "w", encoding="utf-8") as f:
        f.write(_abi())
    os.replace(tmp, _binding_abi_path())


def load_binding():
    """The native binding's module; raises if it is not built, or for another PyTorch or Python."""
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"binding not built: {BINDING_PATH} is missing "
                           "(run exact_attention_55_gb300.build.build())")
    if _binding_abi() != _abi():
        raise RuntimeError(f"{BINDING_PATH} was built against {_binding_abi() or 'an unknown PyTorch'}, here is "
                           f"{_abi()} (run exact_attention_55_gb300.build.build())")
    loader = importlib.machinery.ExtensionFileLoader(BINDING_NAME, BINDING_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader(BINDING_NAME, loader))
    loader.exec_module(module)
    return module


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of the shared library."""
    def fresh(path):
        return not force and os.path.exists(path) and os.path.getmtime(path) >= _sources_mtime()

    if fresh(LIB_PATH):
        if not (fresh(BINDING_PATH) and _binding_abi() == _abi()):
            _compile_binding()
        return LIB_PATH
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_unit(unit):
        name, src, defs = unit
        obj = os.path.join(BUILD, name + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *defs, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.append("-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {name}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(UNITS) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(compile_unit, UNITS))
    if verbose:
        for obj, log in results:
            print(f"== {os.path.basename(obj)}\n{log}")
    objs = [o for o, _ in results]
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    binding.result()                       # the library is there even if this raises
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
