"""The tensor binding (_attn_torch) is apart from the C library: what keeps it from being built or
loaded takes neither the library nor the serving calls with it."""
import os
import sys

import pytest
import torch

from precision_numerics_gb300 import attn, build


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A build of one small source in a folder of its own."""
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "_sources", lambda: [str(tmp_path / "one.cu")])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path / "_lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "_lib" / "libattn.so"))
    return tmp_path


def test_library_without_the_binding(place, monkeypatch):
    """A compiler or headers that fail on the binding are reported; the library is there, is not built
    again, and the binding is tried again."""
    def fail(build_dir):
        raise RuntimeError("g++ on torch_calls.cpp failed: no such header")
    monkeypatch.setattr(build, "_compile_binding", fail)
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert build.build() == build.LIB
    first = os.stat(build.LIB)
    with pytest.warns(RuntimeWarning, match="no such header"):
        build.build()
    assert os.stat(build.LIB).st_mtime_ns == first.st_mtime_ns


def test_library_without_pytorch(place, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # `import torch` raises ImportError
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not build.needs_build()


def test_serving_calls_without_the_binding(tmp_path, monkeypatch):
    """The calls' own checks and the ctypes way do without it."""
    build.build()
    monkeypatch.setattr(attn, "_BINDING", None)
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "missing.so"))
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = [torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 16, 64, dtype=torch.int8),
             torch.zeros(3, 2), torch.zeros(3, 2), torch.zeros(1, 2, dtype=torch.int32)]
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="missing.so"):
        with pytest.raises(ValueError, match="CUDA"):
            attn.attn_varlen_fwd(x, x, x, torch.zeros(512, dtype=torch.uint8))
    for call in (lambda: attn.attn_cache_append_int8(x, x, *cache, ints, ints[:1]),
                 lambda: attn.attn_cache_read_int8(*cache, ints, ints[:1], 4),
                 lambda: attn.attn_decode_int8(x[None], *cache, ints[:1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_serving_calls_give_the_same_without_the_binding(cuda_device, tmp_path, monkeypatch):
    build.build()
    H, Hkv, d, page, T = 4, 2, 64, 16, 70
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, H + 2 * Hkv, d), generator=g).bfloat16().cuda()
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        cache = [torch.zeros((5, Hkv, page, d), dtype=torch.int8, device="cuda") for _ in range(2)]
        cache += [torch.zeros((5, Hkv), device="cuda") for _ in range(2)]
        cache.append(torch.tensor([[3, 1, 0, 4, 2]], dtype=torch.int32, device="cuda"))
        out = [*attn.attn_varlen_fwd(q, k, v, attn.attn_varlen_plan(cu, T, H, Hkv))]
        out += attn.attn_cache_append_int8(k, v, *cache, cu, zero)
        out += attn.attn_cache_read_int8(*cache, cu, zero, T)
        out += attn.attn_decode_int8(q[None, T - 2:], *cache, cu[1:])
        attn.attn_check_status()
        return out

    with_it = run()
    monkeypatch.setattr(attn, "_BINDING", None)
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "missing.so"))
    with pytest.warns(RuntimeWarning, match="missing.so"):
        without = run()
    assert len(with_it) == len(without) == 8
    assert all(torch.equal(a, b) for a, b in zip(with_it, without))
