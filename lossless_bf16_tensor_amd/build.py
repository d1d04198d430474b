"""Build the HIP library libuzip.so in-tree for gfx950 with hipcc."""
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
# the codec, and the KV-cache operators
SRCS = [os.path.join(CSRC, f) for f in ("uzip.hip", "uzip_kv.hip", "uzip_kv_attend.hip")]
LIB = os.path.join(HERE, "libuzip.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no packed-FP32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


# Host code only under AddressSanitizer and UndefinedBehaviorSanitizer (the
# device code is built as usual): for CPU tests of the host-side stream
# parsing, validation and table building. The process that loads such a
# build must preload clang's ASan runtime.
SANITIZE_FLAGS = [
    "-Xarch_host", "-fsanitize=address",
    "-Xarch_host", "-fsanitize=undefined",
    "-Xarch_host", "-fno-sanitize-recover=undefined",
    "-Xarch_host", "-fno-omit-frame-pointer",
    "-g",
]


def _run(cmd: list) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + r.stdout + r.stderr)
    return r.stderr


def build(verbose: bool = False, sanitize: bool = False, out: str | None = None) -> str:
    lib = out or LIB
    flags = [*FLAGS, *(SANITIZE_FLAGS if sanitize else [])]
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(len(SRCS)) as pool:
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SRCS]
        said = list(pool.map(lambda so: _run([HIPCC, *flags, "-I", os.path.join(ROOT, "include"), "-c", so[0], "-o", so[1]]),
                             zip(SRCS, objs)))
        said.append(_run([HIPCC, *flags, "-shared", "-o", lib + ".tmp", *objs]))
    if verbose:
        print("".join(said))
    os.replace(lib + ".tmp", lib)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
