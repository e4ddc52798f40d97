"""Build the CUDA library ``libscem_gmm.so`` in-tree for sm_100a (B200).

nvcc cross-compiles without a GPU, so this also runs on a CPU-only machine.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libscem_gmm.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SOURCES = ["gmm_api.cu", "rows_api.cu", "moe_api.cu", "embed_api.cu", "route_api.cu", "beam_api.cu"]
OBJ = os.path.join(HERE, "_build")  # one object per source
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "gmm.h"))
    return files


def _object(src):
    return os.path.join(OBJ, os.path.splitext(src)[0] + ".o")


def _stale(src):
    """Whether a source's object is missing or older than a file it was made from."""
    obj, deps = _object(src), _object(src)[:-2] + ".d"
    if not (os.path.exists(obj) and os.path.exists(deps)):
        return True
    with open(deps) as f:
        names = f.read().replace("\\\n", " ").split(":", 1)[-1].split()
    made = os.path.getmtime(obj)
    ours = [n for n in names if os.path.abspath(n).startswith(ROOT + os.sep)]
    return not ours or any(not os.path.exists(n) or os.path.getmtime(n) > made for n in ours)


def _command():
    """What the objects come from besides their sources: compiler, version, flags."""
    try:
        version = subprocess.run([NVCC, "--version"], capture_output=True, text=True).stdout
    except OSError:  # (no compiler here: a built library can still be used)
        return None
    return "\n".join([NVCC, version, *FLAGS, *SOURCES])


def _record():
    return os.path.join(OBJ, "command")


def _recorded():
    if not os.path.exists(_record()):
        return None
    with open(_record()) as f:
        return f.read()


def _write_record(text):
    with open(_record(), "w") as f:
        f.write(text)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if it is missing, older than any source, or made by another command.

    (A library that came without the record of its command is taken as it is.)
    """
    now, made_by = _command(), _recorded()
    if not force and os.path.exists(LIB) and (now is None or made_by in (None, now)):
        newest = max(os.path.getmtime(f) for f in _inputs())
        if os.path.getmtime(LIB) >= newest:
            return LIB
    os.makedirs(OBJ, exist_ok=True)
    every = force or made_by != now
    _write_record("unfinished")
    jobs = []
    for src in SOURCES:
        if not every and not _stale(src):
            continue
        obj = _object(src)
        cmd = [NVCC, *(["-Xptxas=-v"] if verbose else []), *FLAGS, "-I", INCLUDE, "-I", CSRC,
               "-MD", "-MF", obj[:-2] + ".d", "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((cmd, subprocess.Popen(cmd)))
    failed = [(cmd, job.returncode) for cmd, job in jobs if job.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(failed[0][1], failed[0][0])
    subprocess.check_call([NVCC, *FLAGS, "-shared", "-o", LIB + ".tmp", *map(_object, SOURCES)])
    os.replace(LIB + ".tmp", LIB)
    _write_record(now)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
