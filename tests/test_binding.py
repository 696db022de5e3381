"""The C API module of the serving calls, by itself: entry points of the C library stand for the
library's, objects with a tensor's attributes for tensors (no GPU is needed)."""
import ctypes
import importlib.util
import os
import shutil
import threading
import time

import pytest

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
