"""Appending a step's rows where requests were left without pages: host-side checks (no kernel is launched)."""
import pytest
import torch

from precision_numerics_gb300 import attn, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


def _append(lib, *, k=16, strides=(128, 64, 128, 64), cache=16, table=16, cu=16, starts=16, lens=16, B=2, T=3, page=16):
    return lib.attn_cache_append_served_int8(k, 16, *strides, cache, 16, 16, 16, table, cu, starts, lens, B, T, 2, 64, 9,
                                             page, 4, None)


def test_arguments(lib):
    """(Without a GPU no pointer passes the checks: those of lens are with the GPU's tests.)"""
    for bad, word in ((dict(cache=8), "k_cache"), (dict(B=0), "B"), (dict(T=-1), "T"),
                      (dict(strides=(128, 63, 128, 64)), "k_head_stride")):
        assert _append(lib, **bad) == attn.ATTN_ERR_INVALID_ARG and word in lib.attn_last_error().decode(), bad
    assert _append(lib, page=48) == attn.ATTN_ERR_UNSUPPORTED


def test_binding_checks_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = [torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 16, 64, dtype=torch.int8),
             torch.zeros(3, 2), torch.zeros(3, 2), torch.zeros(1, 2, dtype=torch.int32)]
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_cache_append_int8(x, x, *cache, ints, ints[:1], lens=ints[:1])
