"""The C API module of the serving calls, by itself: entry points of the C library stand for the
library's, objects with a tensor's attributes for tensors (no GPU is needed)."""
import ctypes
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import threading
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

F16, F32, I32, I64, U8 = (object() for _ in range(5))


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, at=4096):
        self.shape, self.dtype, self.at = tuple(shape), dtype, at

    def stride(self):
        out, n = [], 1
        for x in reversed(self.shape):
            out.insert(0, n)
            n *= x
        return tuple(out)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def module(tmp_path_factory):
    """A copy of the module with statics of its own, every entry point usleep(first argument)."""
    import weight_only_int4_quant_gb300 as tlq

    tlq.build()
    path = str(tmp_path_factory.mktemp("binding") / "_tlq_binding.so")
    shutil.copy(tlq._BINDING_PATH, path)
    spec = importlib.util.spec_from_file_location("_tlq_binding", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    m.bind(F16, F32, I32, I64, U8, lambda: 0, lambda d: 0, *[usleep] * 5)
    return m


MICROSECONDS = 300000


def calls(m):
    """Each of the five with a first argument of MICROSECONDS (a tensor's or the cache's address)."""
    i = lambda *s, at=4096: Tensor(s, I32, at)  # noqa: E731
    h = lambda *s, at=4096: Tensor(s, F16, at)  # noqa: E731
    slots = Tensor((2,), I64)
    return {
        "plan": lambda: m.plan(i(3, at=MICROSECONDS), i(3), i(3, 4), i(9), i(4), i(3), i(2), i(2), slots, i(4), 16, 10,
                               None, None),
        "append": lambda: m.append(MICROSECONDS, 4, 64, h(2, 4, 64), h(2, 4, 64), slots, None),
        "read": lambda: m.read(MICROSECONDS, 4, 64, slots, h(2, 4, 64), h(2, 4, 64), None),
        "attention": lambda: m.attention(MICROSECONDS, 64, h(2, 8, 64), h(2, 8, 64), i(4), i(3), i(3, 4), 1, 0.5, 0,
                                         Tensor((64,), U8), None),
        "lora": lambda: m.lora(h(2, 64, at=MICROSECONDS), h(5, 8, 64), h(5, 32, 8), Tensor((5,), F32), i(4), i(3), 1,
                               h(2, 32), h(2, 32), None),
    }


@pytest.mark.parametrize("name", ["plan", "append", "read", "attention", "lora"])
def test_other_threads_run_during_a_call(module, name):
    call = calls(module)[name]
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.002)

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        time.sleep(0.02)
        begin = time.monotonic()
        assert call() == 0
        end = time.monotonic()
    finally:
        stop.set()
        thread.join()
    assert end - begin >= 0.9e-6 * MICROSECONDS  # the call was made
    assert sum(begin + 0.05 < t < end - 0.05 for t in ticks) > 10


def run_python(code):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)


@pytest.mark.parametrize("missing", ["module", "torch", "both"])
def test_the_library_loads_without_it(module, missing):
    code = "import sys\n" + ("sys.modules['torch'] = None\n" if missing != "module" else "")
    code += "import weight_only_int4_quant_gb300 as tlq\n"
    code += "tlq._BINDING_PATH = '/nowhere.so'\n" if missing != "torch" else ""
    r = run_python(code + "tlq.load(); print(tlq.tl_version(), tlq.tl_kv4_block_bytes(16, 128, 128))")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[-1] == str(16 * (128 + 8))


def test_the_library_builds_without_a_c_compiler(module, tmp_path, monkeypatch):
    import weight_only_int4_quant_gb300 as tlq

    b = sys.modules["weight_only_int4_quant_gb300.build"]
    there = tmp_path / os.path.basename(b.BINDING)
    monkeypatch.setattr(b, "BINDING", str(there))
    for cc in ("no-such-compiler", "false"):
        there.write_bytes(b"of an older source")
        os.utime(there, (1, 1))
        monkeypatch.setenv("CC", cc)
        with pytest.warns(UserWarning, match="C API module"):
            assert tlq.build() == b.LIB
        assert not there.exists()  # an older one does not stay


def test_each_interpreter_has_its_own(module):
    import weight_only_int4_quant_gb300 as tlq

    assert tlq._BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.gpu
def test_the_long_way_gives_the_same(lib, monkeypatch):
    import test_serve_gpu as serve

    torch = serve.torch
    assert lib._short is not lib._LongWay  # built and in use
    short = []
    for way in (lib._short, lib._LongWay):
        monkeypatch.setattr(lib, "_short", way)
        c = serve.Case(lib, [50, 300, 7], [2, 1, 1], 8, 2, 128, 128, 16, seed=3)
        ko, vo = (torch.empty(300, 2, 128, dtype=torch.float16, device="cuda") for _ in "kv")
        slots = c.table[1].long()[torch.arange(300, device="cuda") // 16] * 16 + torch.arange(300, device="cuda") % 16
        lib.tl_kv4_read(c.cache, slots, ko, vo)
        g = torch.Generator("cuda").manual_seed(1)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g).half()  # noqa: E731
        low = lib.lora_add(r(4, 64), r(2, 8, 64), r(2, 32, 8), torch.ones(2, device="cuda"), c.start,
                           torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda"), 2, r(4, 32))
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        plan = [i32(4), i32(3), i32(5), i32(5), torch.zeros(5, dtype=torch.int64, device="cuda"), i32(4)]
        lib.tl_kv_plan(i32(3), torch.tensor([2, 1, 1], dtype=torch.int32, device="cuda"), c.table.clone(),
                       torch.arange(9, dtype=torch.int32, device="cuda"), *plan, page_size=16, num_pages=40)
        short.append([c.run(lib, 0.1), ko, vo, low, *plan])
    for a, b in zip(*short):
        assert torch.equal(a, b)
