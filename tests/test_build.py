"""CPU: what an interrupted or failed compilation leaves behind does not pass
for a finished one."""
import importlib.util
import os
import stat

import pytest

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# by its file: the package around it wants the library that it builds
spec = importlib.util.spec_from_file_location("mqc_build", os.path.join(HERE, "im2col_gemm_b200", "build.py"))
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)


def test_an_unfinished_dependency_list_is_not_up_to_date(tmp_path):
    obj = tmp_path / "unit.o"
    for text in ("", "unit.o", "unit.o :", "unit.o: \\\n"):
        (tmp_path / "unit.o.d").write_text(text)
        obj.write_text("")
        assert not b.object_up_to_date(str(obj)), repr(text)
    (tmp_path / "unit.cu").write_text("")
    os.utime(tmp_path / "unit.cu", (1, 1))
    (tmp_path / "unit.o.d").write_text(f"{obj} : {tmp_path / 'unit.cu'}\n")
    assert b.object_up_to_date(str(obj))


def test_a_failed_unit_leaves_the_others_and_its_own_past(tmp_path, monkeypatch):
    """The compiler writes the dependency list before it is done: the list of a
    unit that fails must not replace the one that belongs to its object."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do case "$1" in -MF) d="$2";; -o) o="$2";; esac; last="$1"; shift; done\n'
                    'echo "half" > "$d"\ncase "$last" in *linear.cu) exit 1;; esac\necho new > "$o"\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    objects = tmp_path / "objects"
    objects.mkdir()
    for name in ("linear.o", "linear.o.d", "dropout.o", "dropout.o.d"):
        (objects / name).write_text("old\n")
    for name, value in (("NVCC", str(nvcc)), ("OBJ", str(objects)), ("LIB", str(tmp_path / "lib.so"))):
        monkeypatch.setattr(b, name, value)
    with pytest.raises(Exception, match="linear"):
        b.build(force=True)
    assert (objects / "linear.o").read_text() == (objects / "linear.o.d").read_text() == "old\n"
    assert (objects / "dropout.o").read_text() == "new\n" and (objects / "dropout.o.d").read_text() == "half\n"
    assert not [f for f in os.listdir(objects) if "tmp" in f] and not os.path.exists(tmp_path / "lib.so")
