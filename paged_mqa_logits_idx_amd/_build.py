"""Build step (in-tree) for the HIP libraries (gfx950): libidx_paged_mqa.so, the
indexer and its caches, and libidx_read_stream.so, the bare key-page read stream that the
benchmark measures as the reachable HBM read rate; and for _binding.so, the host code
that marshals tensors for the former."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG_DIR = Path(__file__).resolve().parent
REPO_DIR = PKG_DIR.parent
SOURCES = [PKG_DIR / "csrc" / name for name in ("paged_mqa_logits.hip", "norm_rope.hip", "latent_attention.hip",
                                                "kv_cache.hip", "kv_attention.hip")]
LIB_PATH = PKG_DIR / "libidx_paged_mqa.so"
STREAM_SOURCES = [PKG_DIR / "csrc" / "read_stream.hip"]
STREAM_LIB_PATH = PKG_DIR / "libidx_read_stream.so"
BINDING_SOURCE = PKG_DIR / "csrc" / "binding.cpp"
BINDING_PATH = PKG_DIR / "_binding.so"
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("hipcc not found: the HIP library cannot be built")


def build_command(out: Path = LIB_PATH, sources=None) -> list[str]:
    return [
        hipcc(),
        f"--offload-arch={ARCH}",
        "-O3",
        "-std=c++17",
        "-shared",
        "-fPIC",
        # packed fp32 VALU ops are kept out of every kernel
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        f"-I{REPO_DIR / 'include'}",
        *[str(s) for s in (SOURCES if sources is None else sources)],
        "-o", str(out),
    ]


def binding_command(out: Path = BINDING_PATH) -> list[str]:
    """Host code against torch's and Python's headers; what it needs of torch's
    libraries is loaded with torch."""
    import torch

    home = Path(torch.__file__).resolve().parent
    rocm = Path(hipcc()).resolve().parent.parent
    return [
        shutil.which("g++") or "g++",
        "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
        f"-I{REPO_DIR / 'include'}",
        *[f"-isystem{d}" for d in (sysconfig.get_paths()["include"], home / "include",
                                   home / "include" / "torch" / "csrc" / "api" / "include", rocm / "include")],
        str(BINDING_SOURCE),
        f"-L{home / 'lib'}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python",
        "-o", str(out),
    ]


def build(verbose: bool = False) -> Path:
    """Compile all of it; always recompiles.  Writes atomically."""
    with ThreadPoolExecutor(3) as pool:
        made = [pool.submit(_compile, lib, command(lib.with_name(lib.name + ".tmp")), verbose) for lib, command in (
            (LIB_PATH, build_command), (STREAM_LIB_PATH, lambda out: build_command(out, STREAM_SOURCES)),
            (BINDING_PATH, binding_command))]
        return [m.result() for m in made][0]


def _compile(lib: Path, cmd: list[str], verbose: bool) -> Path:
    tmp = lib.with_name(lib.name + ".tmp")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        out = (res.stdout + res.stderr).strip()
        # hipcc's host pass does not know the packed-fp32 feature; drop that noise
        out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l)
        if out:
            print(out)
    if res.returncode != 0:
        raise RuntimeError(f"the compiler failed ({res.returncode}): {' '.join(cmd)}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
