"""How the C API module reads torch's tensors: the same answers as through their attributes."""
import ctypes
import importlib.util
import os
import shutil

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def tlq():
    import weight_only_int4_quant_gb300 as tlq

    tlq.build()
    tlq.load()
    return tlq


def test_built_for_this_torch_or_not_at_all(tlq, tmp_path, monkeypatch):
    import sys

    b = sys.modules["weight_only_int4_quant_gb300.build"]
    if not b.build_tensors():
        pytest.skip("torch's headers are not there")
    assert open(b.TENSORS_OF).read() == torch.__version__
    lib = ctypes.CDLL(b.TENSORS)
    lib.tlq_torch_version.restype = ctypes.c_char_p
    assert torch.__version__.split("+")[0] == lib.tlq_torch_version().decode().split("+")[0]
    # another torch's is not used
    other = tmp_path / "of.torch"
    other.write_text("0.1")
    monkeypatch.setattr(tlq, "_TENSORS_OF", str(other))

    class Module:
        @staticmethod
        def read_tensors(*args):
            raise AssertionError("used")

    tlq._read_tensors(Module)
    # and without a compiler there is none, an older one included
    for name in ("TENSORS", "TENSORS_OF"):
        path = tmp_path / name
        path.write_text("old")
        monkeypatch.setattr(b, name, str(path))
    monkeypatch.setenv("CXX", "false")
    assert not b.build_tensors(force=True)
    assert not (tmp_path / "TENSORS").exists() and not (tmp_path / "TENSORS_OF").exists()


@pytest.mark.gpu
def test_the_same_as_by_attributes(lib, tmp_path):
    """Good and bad arguments through a copy of the module that does not read tensors directly and through the one
    in use: the same answers, the same results."""
    path = str(tmp_path / "_tlq_binding.so")
    shutil.copy(lib._BINDING_PATH, path)
    spec = importlib.util.spec_from_file_location("_tlq_binding", path)
    plain = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(plain)
    types = (torch.float16, torch.float32, torch.int32, torch.int64, torch.uint8)
    at = lambda *names: [ctypes.cast(getattr(lib.load(), n), ctypes.c_void_p).value for n in names]  # noqa: E731
    plain.bind(*types, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream,
               *at("tl_kv_plan", "tl_kv4_append", "tl_kv4_read", "tl_kv4_attention", "tl_lora_add"))
    plain.bind_step(*at("tl_qk_norm_rope", "tl_kv4_append_rope", "tl_sample", "tl_kv4_attention_prefix"))
    g = torch.Generator("cuda").manual_seed(0)
    rows = torch.randn(6, 5, 64, device="cuda", generator=g).half()
    odd = [rows, rows[:, 1:4], rows[:, :, ::2], rows.transpose(0, 1), rows[:1, 2:5], rows[::2, 1:4], rows[:0], rows.float(),
           rows.cpu(), torch.nn.Parameter(rows), rows.view(6, 320), rows[0], rows.bfloat16(), None, 3, "x",
           torch.empty(6, 5, 64, dtype=torch.float16, device="meta"), rows.expand(6, 5, 64), rows[:1].expand(6, 5, 64),
           torch.sparse_coo_tensor(torch.zeros(1, 1, dtype=torch.int64), torch.ones(1, 5, 64), (6, 5, 64), device="cuda")]
    for x in odd:
        answers = []
        for m in (plain, lib._short):
            like = isinstance(x, torch.Tensor) and x.dim() == 3 and x.is_cuda and x.layout is torch.strided
            out = torch.zeros(x.shape, dtype=torch.float16, device="cuda") if like else None
            answers.append((m.norm_rope(None, 0, x, None, None, out, None, None, None, 1e-6, None), out))
        assert answers[0][0] == answers[1][0], x
        assert answers[0][1] is None or torch.equal(answers[0][1], answers[1][1])
        if answers[0][0] == 0:
            assert torch.equal(answers[0][1], x.detach())
    u = torch.rand(6, device="cuda")
    logits = torch.randn(6, 40, device="cuda")
    for x, s in ((logits, u), (logits.half(), u), (logits.t(), u), (logits[:, ::2], u), (logits[:, :7], u), (logits, u.half()),
                 (logits, u[:5]), (logits, u[::2]), (logits.double(), u), (logits[0], u), (logits, u.cpu()),
                 (logits, torch.nn.Parameter(u))):
        got = []
        for m in (plain, lib._short):
            t = torch.full((6,), -5, dtype=torch.int32, device="cuda")
            got.append((m.sample(x, s, t, None, None, None, None, None, None), t.tolist()))
        assert got[0] == got[1]
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_tensors_that_stand_for_others_are_refused(lib):
    """Inside torch.func's transforms tensors have no storage: an error, not the end of the process."""
    u = torch.rand(6, device="cuda")
    logits = torch.randn(3, 6, 40, device="cuda")
    tokens = torch.full((6,), -5, dtype=torch.int32, device="cuda")
    rows = torch.randn(3, 6, 5, 64, device="cuda").half()
    out = torch.zeros(6, 5, 64, dtype=torch.float16, device="cuda")

    def draw(x):
        lib.tl_sample(x, u, tokens)
        return x.sum()

    def norm(x):
        lib.tl_qk_norm_rope(None, x, None, None, out, None)
        return x.float().sum()

    for f, x in ((draw, logits), (norm, rows)):
        with pytest.raises(RuntimeError):
            torch.func.vmap(f)(x)
        with pytest.raises(RuntimeError):
            torch.func.grad(f)(x[0])
    torch.cuda.synchronize()
    assert tokens.tolist() == [-5] * 6 and not out.any()
