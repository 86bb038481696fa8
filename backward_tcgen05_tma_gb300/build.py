"""Builds libswiglu_mlp.so (release) and libswiglu_mlp_debug.so (the same
sources with -DSWIGLU_DEBUG: device index checks) in place with nvcc for
sm_103a (GB300).  The two compile in parallel."""
from __future__ import annotations

import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
CSRC_SERVING = os.path.join(HERE, "csrc_serving")
CSRC_BLOCK = os.path.join(HERE, "csrc_block")
ROOT = os.path.dirname(HERE)
SO = os.path.join(HERE, "libswiglu_mlp.so")
SO_DEBUG = os.path.join(HERE, "libswiglu_mlp_debug.so")
BUILD = os.path.join(HERE, "_build")  # objects, kept for the next build

# translation units
SOURCES = [
    os.path.join(CSRC, "swiglu_mlp.cu"),
    os.path.join(CSRC_SERVING, "serving.cu"),
    os.path.join(CSRC_BLOCK, "block.cu"),
]

NVCC_FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-Xcompiler", "-fPIC",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _includes(path: str, found: set[str]) -> set[str]:
    """path and the files that its quoted includes lead to (each is looked for
    beside the file that names it)."""
    path = os.path.normpath(path)
    if path not in found and os.path.exists(path):
        found.add(path)
        with open(path) as f:
            for name in re.findall(r'^[ \t]*#[ \t]*include[ \t]+"([^"]+)"', f.read(), re.M):
                _includes(os.path.join(os.path.dirname(path), name), found)
    return found


def _deps(src: str) -> list[str]:
    return sorted(_includes(src, set())) + [os.path.abspath(__file__)]


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmds) -> None:
    """Runs the commands ([argv, output]) at the same time, each into a file of
    its own that then takes its output's place; raises if one fails."""
    procs = []
    for cmd, out in cmds:
        tmp = "%s.%d.tmp" % (out, os.getpid())
        procs.append((subprocess.Popen(cmd + ["-o", tmp]), cmd, tmp, out))
    failed = None
    for p, cmd, tmp, out in procs:
        if p.wait() != 0:
            failed = failed or subprocess.CalledProcessError(p.returncode, cmd)
            if os.path.exists(tmp):
                os.remove(tmp)
        else:
            os.replace(tmp, out)
    if failed is not None:
        raise failed


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile whichever objects and libraries are missing or out of date (the
    objects in parallel); returns the release library's path."""
    os.makedirs(BUILD, exist_ok=True)
    compiles, links = [], []
    for so, name, extra in ((SO, "release", []), (SO_DEBUG, "debug", ["-DSWIGLU_DEBUG"])):
        objs = []
        for src in SOURCES:
            obj = os.path.join(BUILD, "%s_%s.o" % (os.path.basename(src)[:-3], name))
            objs.append(obj)
            if force or _stale(obj, _deps(src)):
                compiles.append(([_nvcc(), *NVCC_FLAGS, *extra, "-c", src], obj))
        links.append(([_nvcc(), *NVCC_FLAGS, "-shared", *objs], so, objs))
    if verbose:
        for cmd, _ in compiles:
            print(" ".join(cmd))
    _run(compiles)
    _run([(cmd, so) for cmd, so, objs in links if force or _stale(so, objs)])
    return SO


if __name__ == "__main__":
    print(build(force=True, verbose=True))
