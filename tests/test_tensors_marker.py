"""The reader of torch's tensors is never taken for one of another torch, whenever its build stops."""
import importlib
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

COMPILER = """#!%s
import sys
open(sys.argv[sys.argv.index("-o") + 1], "w").write("new")
"""


@pytest.fixture
def b(tmp_path, monkeypatch):
    """The build module with its reader's two files in a folder of their own, and a compiler that only writes its output."""
    import weight_only_int4_quant_gb300  # noqa: F401

    b = sys.modules["weight_only_int4_quant_gb300.build"]
    root = os.path.dirname(importlib.util.find_spec("torch").origin)
    if not os.path.exists(os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h")):
        pytest.skip("torch's headers are not there")
    for name, text in (("TENSORS", "old"), ("TENSORS_OF", torch.__version__)):
        path = tmp_path / name
        path.write_text(text)
        monkeypatch.setattr(b, name, str(path))
    cxx = tmp_path / "cxx"
    cxx.write_text(COMPILER % sys.executable)
    cxx.chmod(0o755)
    monkeypatch.setenv("CXX", str(cxx))
    return b


def read(path):
    return open(path).read() if os.path.exists(path) else None


def test_a_stopped_build_leaves_no_marker_beside_the_new_reader(b, monkeypatch):
    """At every step that changes a file: the marker stands only beside the reader it was written for."""
    whole = {name: getattr(os, name) for name in ("replace", "remove")}
    steps = []

    class Stop(Exception):
        pass

    for stop in range(8):
        for path, text in ((b.TENSORS, "old"), (b.TENSORS_OF, "of the old")):
            with open(path, "w") as f:
                f.write(text)
        steps.clear()

        def step(name):
            def f(*args):
                whole[name](*args)
                steps.append(name)
                if len(steps) == stop + 1:
                    raise Stop
            return f

        for name in whole:
            monkeypatch.setattr(os, name, step(name))
        try:
            done = b.build_tensors(force=True)
        except Stop:
            done = None
        for name, f in whole.items():
            monkeypatch.setattr(os, name, f)
        pair = read(b.TENSORS), read(b.TENSORS_OF)
        assert pair in (("old", "of the old"), ("old", None), ("new", None), ("new", torch.__version__)), (stop, pair)
        if done is not None:
            assert done and pair == ("new", torch.__version__)
            return
    raise AssertionError("the build does not end")


def test_the_marker_is_never_half_written(b, monkeypatch):
    """It comes by one rename: nothing opens it for writing in its place."""
    written = []
    plain = open

    def watch(path, mode="r", *args, **k):
        if "w" in mode:
            written.append(str(path))
        return plain(path, mode, *args, **k)

    monkeypatch.setattr(b, "open", watch, raising=False)
    assert b.build_tensors(force=True)
    assert read(b.TENSORS_OF) == torch.__version__ and b.TENSORS_OF not in written


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_the_reader_says_itself_what_it_was_built_for(tmp_path, monkeypatch):
    import weight_only_int4_quant_gb300 as tlq

    marker = tmp_path / "of.torch"
    marker.write_text(torch.__version__)
    monkeypatch.setattr(tlq, "_TENSORS_OF", str(marker))
    used = []

    class Module:
        @staticmethod
        def read_tensors(*args):
            used.append(args)

    own = torch.__version__.split("+")[0]
    for i, (body, taken) in enumerate([('const char* tlq_torch_version(void) { return "%s"; }' % own, True),
                                       ('const char* tlq_torch_version(void) { return "0.1.2"; }', False),
                                       ("", False)]):
        src, so = tmp_path / ("r%d.c" % i), tmp_path / ("r%d.so" % i)
        src.write_text(body + "\nint tlq_tensor_read(void* o, void* t) { return 0; }\n")
        subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
        monkeypatch.setattr(tlq, "_TENSORS_PATH", str(so))
        used.clear()
        tlq._read_tensors(Module)
        assert bool(used) == taken, body
