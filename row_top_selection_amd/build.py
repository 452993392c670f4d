"""Ahead-of-time build of libdsatopk.so for gfx950 with hipcc, and of the
serving operators' Python calls with g++ (both in-tree)."""
from __future__ import annotations

import os
import subprocess
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
SOURCES = [PKG / "csrc" / name for name in (
    "dsatopk.hip", "page_maps.hip", "append_cache.hip", "index_scores.hip", "latent_attend.hip",
    "shared_attend.hip", "expanded_attend.hip")]
HEADERS = [PKG / "csrc" / "select_device.h", PKG / "csrc" / "serve_common.h",
           PKG / "csrc" / "latent_tiles.h", PKG / "csrc" / "wide_tiles.h",
           ROOT / "include" / "dsatopk.h"]
LIB = PKG / "libdsatopk.so"
EXT_SOURCE = PKG / "csrc" / "serve_binding.cpp"
EXT = PKG / ("_serve" + sysconfig.get_config_var("EXT_SUFFIX"))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -packed-fp32-ops: keep the compiler from forming packed fp32 instructions.
FLAGS = [
    "-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", str(ROOT / "include"),
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode}):\n{res.stderr}")


def _build_ext(verbose):
    """The extension module, against the torch that is installed."""
    from torch.utils import cpp_extension

    tmp = EXT.with_suffix(".so.tmp%d" % os.getpid())
    rocm = Path(HIPCC).resolve().parents[1]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
           "-DUSE_ROCM", "-I", str(ROOT / "include")]
    for path in (*cpp_extension.include_paths(), str(rocm / "include"),
                 sysconfig.get_paths()["include"]):
        cmd += ["-isystem", path]
    cmd += [str(EXT_SOURCE), "-o", str(tmp), "-L", str(PKG), "-ldsatopk", "-Wl,-rpath,$ORIGIN"]
    for path in cpp_extension.library_paths():
        cmd += ["-L", path]
    cmd += ["-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10_hip", "-lc10", "-lamdhip64"]
    _run(cmd, verbose)
    os.replace(tmp, EXT)


def build(force: bool = True, verbose: bool = False) -> Path:
    """Compile every HIP source into ``libdsatopk.so`` next to this file
    (the sources side by side, then one link), and the extension module."""
    newest = max(p.stat().st_mtime for p in [*SOURCES, *HEADERS, EXT_SOURCE])
    if not force and all(p.exists() and p.stat().st_mtime >= newest for p in (LIB, EXT)):
        return LIB
    tmp = LIB.with_suffix(".so.tmp%d" % os.getpid())
    with tempfile.TemporaryDirectory() as d:
        objects = [Path(d) / (p.stem + ".o") for p in SOURCES]
        cmds = [[HIPCC, *FLAGS, "-c", str(p), "-o", str(o)] for p, o in zip(SOURCES, objects)]
        with ThreadPoolExecutor(max_workers=min(8, len(cmds))) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), cmds))
        _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *map(str, objects), "-o",
              str(tmp)], verbose)
    os.replace(tmp, LIB)
    _build_ext(verbose)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
