"""Build libtdi8.so (gfx950) in-tree with hipcc.

One object per tile configuration (instantiate.hip compiled with
-DTDI8_CFG=<id>), plus the host selection and the C-ABI dispatcher, linked
into tiled_dense_int8_amd/libtdi8.so.  Objects go to _build/ at the repo root.

Between compiling and linking, the register and LDS use of every
configuration's column-major kernel (the one the selection's occupancy is
taken on) is read from the AMDGPU metadata note of the gfx950 code object
this build just produced, and compiled into the library as a table
(_build/kernel_resources.cpp): tile_config_info reports it.  The same file
carries the SHA-256 of those code objects (tdi8_kernel_code_hash) and that of
the 8-bit layer operators' (tdi8_layer_code_hash).

The library build also produces libtdi8_ceilings.so (roofline calibration
kernels) and libtdi8_stamps.so: the same sources compiled with TDI8_STAMPS,
whose kernels write per-block timelines (include/tdi8_stamps.h); its
objects go to _build/stamps/.  _calls.so is the Python module of the 8-bit
layer operators' ordinary calls (csrc/calls.cpp), host code against torch's
headers.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

import yaml

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtdi8.so")
CEILINGS_LIB = os.path.join(PKG, "libtdi8_ceilings.so")  # roofline calibration kernels (bench.py --ceilings)
CALLS_LIB = os.path.join(PKG, "_calls.so")                 # ordinary calls of the layer operators
STAMPS_LIB = os.path.join(PKG, "libtdi8_stamps.so")      # block timelines (bench.py --stamps)
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
LLVM_BIN = "/opt/rocm/llvm/bin"
ARCH = "gfx950"

FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 instructions are not wanted in any kernel of this library
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC, "-Wall", "-Wno-unused-function",
]


def config_ids() -> list[int]:
    text = open(os.path.join(CSRC, "configs.h")).read()
    return [int(m) for m in re.findall(r"^\s*X\((\d+),", text, flags=re.M)]


def config_params() -> dict[int, tuple[int, ...]]:
    """id -> (family, MF, WM, WN, WK, MT, NT, BK, ST) from configs.h."""
    text = open(os.path.join(CSRC, "configs.h")).read()
    out = {}
    for m in re.finditer(r"^\s*X\(([\d,\s]+)\)", text, flags=re.M):
        v = [int(x) for x in m.group(1).split(",")]
        out[v[0]] = tuple(v[1:])
    return out


def _run(cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("build step failed: " + " ".join(cmd[-3:]))
    return r.stdout


def occupancy_kernel_symbol(params: tuple[int, ...]) -> str:
    """Mangled name of a configuration's column-major-B unpredicated kernel
    (kernel_table.h: kernel[1][1]), whose resources set its occupancy."""
    fam, mf, wm, wn, wk, mt, nt, bk, st = params
    if fam == 0:
        args = "".join(f"Li{v}E" for v in (mf, wm, wn, mt, nt, bk, st)) + "Lb0ELb0ELb0E"
        return f"_ZN4tdi824gemm_rc_pipelined_kernelI{args}EEvNS_8GemmArgsE"
    args = "".join(f"Li{v}E" for v in (mt, nt, wk, bk))
    return f"_ZN4tdi822gemm_skinny_lds_kernelI{args}EEvNS_8GemmArgsE"


def code_object_path(obj: str, work: str) -> str:
    return os.path.join(work, os.path.basename(obj) + ".co")


def extract_code_object(obj: str, work: str) -> str:
    """The gfx950 code object embedded in a host object built here, as a file
    at code_object_path(obj, work)."""
    fatbin = os.path.join(work, os.path.basename(obj) + ".fatbin")
    co = code_object_path(obj, work)
    _run([os.path.join(LLVM_BIN, "llvm-objcopy"), f"--dump-section=.hip_fatbin={fatbin}", obj,
          os.path.join(work, os.path.basename(obj) + ".stripped")])
    _run([os.path.join(LLVM_BIN, "clang-offload-bundler"), "--unbundle", "--type=o",
          f"--targets=hipv4-amdgcn-amd-amdhsa--{ARCH}", f"--input={fatbin}", f"--output={co}"])
    return co


def code_object_kernels(obj: str, work: str) -> dict[str, dict]:
    """Kernel name -> metadata (.vgpr_count, .agpr_count, ...) of an object's
    code object."""
    co = extract_code_object(obj, work)
    notes = _run([os.path.join(LLVM_BIN, "llvm-readelf"), "--notes", co])
    start = notes.index("---")
    end = notes.index("\n...", start)
    meta = yaml.safe_load(notes[start:end])
    return {k[".name"]: k for k in meta["amdhsa.kernels"]}


# The objects of the 8-bit layer operators' kernels, in the order of their hash.
LAYER_OBJECTS = tuple(f"quant_rows_{ty}" for ty in ("F32", "Bf16", "F16")) + \
    tuple(f"stream_{ty}" for ty in ("S8", "F8", "F8Wide")) + ("grouped_tiles", "block_scale_tiles")


def layer_code_hash(bdir: str) -> str:
    code = hashlib.sha256()
    for name in LAYER_OBJECTS:
        with open(extract_code_object(os.path.join(bdir, name + ".o"), bdir), "rb") as f:
            code.update(f.read())
    return code.hexdigest()[:16]


def write_resource_table(objs: dict[int, str], bdir: str) -> str:
    """Generate the C++ table of per-configuration kernel resources, and the
    hashes of the code objects."""
    params = config_params()
    rows = []
    code = hashlib.sha256()
    for cid in sorted(params):
        kernels = code_object_kernels(objs[cid], bdir)
        sym = occupancy_kernel_symbol(params[cid])
        if sym not in kernels:
            raise RuntimeError(f"configuration {cid}: kernel {sym} not found in {objs[cid]}")
        k = kernels[sym]
        with open(code_object_path(objs[cid], bdir), "rb") as f:
            code.update(f.read())
        rows.append(f"    {{{k['.vgpr_count']}, {k['.agpr_count']}, {k['.sgpr_count']}, "
                    f"{k['.group_segment_fixed_size']}, {k['.private_segment_fixed_size']}}},  // {cid}")
    src = os.path.join(bdir, "kernel_resources.cpp")
    text = ("// Generated by tiled_dense_int8_amd/build.py from the AMDGPU metadata of the\n"
            "// gfx950 code objects of this build: resources of each configuration's\n"
            "// column-major-B unpredicated kernel.\n"
            '#include "kernel_table.h"\n\nnamespace tdi8 {\n\n'
            "const KernelResources kKernelResources[TDI8_NUM_CONFIGS] = {\n" + "\n".join(rows) +
            "\n};\n\n}  // namespace tdi8\n\n"
            "// SHA-256 of the code objects of every configuration, in id order.\n"
            'extern "C" const char *tdi8_kernel_code_hash(void) { return "' + code.hexdigest()[:16] + '"; }\n'
            "// The same of the 8-bit layer operators' kernels.\n"
            'extern "C" const char *tdi8_layer_code_hash(void) { return "' + layer_code_hash(bdir) + '"; }\n')
    with open(src, "w") as f:
        f.write(text)
    return src


def calls_unit(out: str) -> list[str]:
    """The command that builds the Python module _calls (host code)."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    include = os.path.join(torch_dir, "include")
    # as torch.__version__ says it, without importing torch
    with open(os.path.join(torch_dir, "version.py")) as f:
        version = re.search(r"^__version__ = '([^']+)'", f.read(), flags=re.M).group(1)
    return [CXX, f'-DTDI8_TORCH_VERSION="{version}"', "-O2", "-std=c++17", "-fPIC", "-shared",
            "-fvisibility=hidden", "-Wall", "-I", INCLUDE,
            "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "calls.cpp"),
            "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", out]


def build(jobs: int | None = None, verbose: bool = False, extra_flags: list[str] | None = None,
          out: str | None = None, build_dir: str | None = None) -> str:
    """Compile every configuration and link the library (default: in-tree libtdi8.so)."""
    out = out or LIB
    bdir = build_dir or BUILD
    flags = FLAGS + list(extra_flags or [])
    os.makedirs(bdir, exist_ok=True)
    jobs = jobs or min(16, os.cpu_count() or 4)
    units = []
    for cid in config_ids():
        obj = os.path.join(bdir, f"cfg{cid}.o")
        units.append([HIPCC, *flags, f"-DTDI8_CFG={cid}", "-c",
                      os.path.join(CSRC, "instantiate.hip"), "-o", obj])
    units.append([HIPCC, *flags, "-x", "hip", "-c", os.path.join(CSRC, "abi.cpp"),
                  "-o", os.path.join(bdir, "abi.o")])
    units.append([HIPCC, *flags, "-x", "hip", "-c", os.path.join(CSRC, "selector.cpp"),
                  "-o", os.path.join(bdir, "selector.o")])
    # the 8-bit layer operators: entry points and the choice of a product's
    # kernel, the row kernels by type, the scaled products by operand type
    for name in ("layer_ops", "product_choice"):
        units.append([HIPCC, *flags, "-x", "hip", "-c", os.path.join(CSRC, name + ".cpp"),
                      "-o", os.path.join(bdir, name + ".o")])
    for ty in ("F32", "Bf16", "F16"):
        units.append([HIPCC, *flags, f"-DTDI8_ROWS_TYPE={ty}", f"-DTDI8_ROWS_REGISTER=register_rows_{ty.lower()}",
                      "-c", os.path.join(CSRC, "quant_rows.hip"), "-o", os.path.join(bdir, f"quant_rows_{ty}.o")])
    for ty in ("S8", "F8", "F8Wide"):
        units.append([HIPCC, *flags, f"-DTDI8_PRODUCT_TYPE={ty}",
                      f"-DTDI8_PRODUCT_REGISTER=register_products_{ty.lower()}",
                      "-c", os.path.join(CSRC, "stream_product.hip"), "-o", os.path.join(bdir, f"stream_{ty}.o")])
    for name in ("grouped_tiles", "block_scale_tiles"):
        units.append([HIPCC, *flags, "-c", os.path.join(CSRC, name + ".hip"), "-o", os.path.join(bdir, name + ".o")])
    ceil_obj = os.path.join(bdir, "ceilings.o")
    ceil_unit = [HIPCC, *flags, "-c", os.path.join(CSRC, "ceilings.hip"), "-o", ceil_obj]
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        calls_tmp = CALLS_LIB + ".tmp%d" % os.getpid()
        list(ex.map(_run, ([calls_unit(calls_tmp), ceil_unit] if out == LIB else []) + units))
    objs = [u[u.index("-o") + 1] for u in units]
    res_src = write_resource_table({cid: os.path.join(bdir, f"cfg{cid}.o") for cid in config_ids()}, bdir)
    res_obj = os.path.join(bdir, "kernel_resources.o")
    _run([HIPCC, *flags, "-c", res_src, "-o", res_obj])
    objs.append(res_obj)
    tmp = out + ".tmp%d" % os.getpid()
    _run([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp])
    os.replace(tmp, out)
    if out == LIB:
        os.replace(calls_tmp, CALLS_LIB)
        tmp = CEILINGS_LIB + ".tmp%d" % os.getpid()
        _run([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", ceil_obj, "-o", tmp])
        os.replace(tmp, CEILINGS_LIB)
        build(jobs, verbose, list(extra_flags or []) + ["-DTDI8_STAMPS"], STAMPS_LIB, os.path.join(bdir, "stamps"))
    if verbose:
        print("built", out)
    return out


if __name__ == "__main__":
    build(verbose=True)
