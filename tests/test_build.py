"""build.build() compiles what is out of date, and all of it when the command changes (CPU; a
script stands in for the compiler)."""
import os
import stat

import pytest

from soft_clustering_em_b200 import build as B

NVCC = """#!/bin/sh
# writes its -o and -MF files and notes the source it was given
if [ "$1" = --version ]; then cat "$0.version"; exit 0; fi
src=link
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out=$2; shift;;
    -MF) dep=$2; shift;;
    -c) src=$(basename "$2");;
  esac
  shift
done
echo "$src" >> "$(dirname "$0")/calls"
echo x > "$out"
if [ -n "$dep" ]; then echo "$out: $(dirname "$0")/csrc/$src $(dirname "$0")/csrc/both.h" > "$dep"; fi
"""


@pytest.fixture()
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("a.cu", "b.cu", "both.h"):
        (csrc / name).write_text("//\n")
    (tmp_path / "gmm.h").write_text("//\n")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(NVCC)
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    (tmp_path / "nvcc.version").write_text("1\n")
    for name, value in dict(ROOT=str(tmp_path), CSRC=str(csrc), INCLUDE=str(tmp_path),
                            OBJ=str(tmp_path / "_build"), LIB=str(tmp_path / "lib.so"),
                            NVCC=str(nvcc), SOURCES=["a.cu", "b.cu"], FLAGS=["-O3"]).items():
        monkeypatch.setattr(B, name, value)
    for f in [csrc / n for n in os.listdir(csrc)] + [tmp_path / "gmm.h"]:
        os.utime(f, (1, 1))

    def calls():
        log = tmp_path / "calls"
        done = sorted(log.read_text().split()) if log.exists() else []
        log.write_text("")
        return done

    return tmp_path, calls


ALL = ["a.cu", "b.cu", "link"]


def test_only_what_is_out_of_date(tree):
    root, calls = tree
    B.build()
    assert calls() == ALL
    B.build()
    assert calls() == []
    later = os.path.getmtime(root / "lib.so") + 10
    os.utime(root / "csrc" / "b.cu", (later, later))
    B.build()
    assert "a.cu" not in calls()
    B.build(force=True)
    assert calls() == ALL


def test_other_flags_compile_everything(tree, monkeypatch):
    _, calls = tree
    B.build()
    calls()
    monkeypatch.setattr(B, "FLAGS", ["-O3", "-lineinfo"])
    B.build()
    assert calls() == ALL
    B.build()
    assert calls() == []


def test_another_compiler_compiles_everything(tree):
    root, calls = tree
    B.build()
    calls()
    (root / "nvcc.version").write_text("2\n")
    B.build()
    assert calls() == ALL
    B.build()
    assert calls() == []


def test_another_source_is_linked(tree, monkeypatch):
    root, calls = tree
    B.build()
    calls()
    monkeypatch.setattr(B, "SOURCES", ["a.cu"])
    B.build()
    assert "link" in calls()


def test_a_build_that_failed_is_done_again(tree, monkeypatch):
    root, calls = tree
    B.build()
    calls()
    monkeypatch.setattr(B, "FLAGS", ["-O2"])
    (root / "nvcc").write_text(NVCC.replace("#!/bin/sh", "#!/bin/sh\n[ $1 = --version ] || exit 1"))
    with pytest.raises(Exception):
        B.build()
    monkeypatch.setattr(B, "FLAGS", ["-O3"])
    (root / "nvcc").write_text(NVCC)
    B.build()
    assert calls() == ALL


def test_a_library_without_a_record_or_a_compiler_is_taken_as_it_is(tree, monkeypatch):
    root, calls = tree
    B.build()
    calls()
    (root / "_build" / "command").unlink()
    B.build()
    assert calls() == []
    monkeypatch.setattr(B, "NVCC", str(root / "none"))
    B.build()
    assert calls() == []
