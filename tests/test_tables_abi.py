"""Block tables and the shared prefix: host-side checks (no kernel is launched), and the plain form of the tables."""
import ctypes

import pytest
import torch

import serving_ref as ref
from precision_numerics_gb300 import attn, build

F = ctypes.c_float
BAD, NO = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


def _reserve(lib, *, table=0x10000, held=0x20000, wanted=0x30000, pages=0x40000, free=0x50000, lens=0x60000, cu=0x70000,
             slots=0x80000, positions=0x90000, B=2, T=40, num_pages=9, page=16, blocks=4):
    return lib.attn_cache_reserve(table, held, wanted, pages, free, lens, cu, slots, positions, B, T, num_pages, page,
                                  blocks, None)


def test_reserve_arguments(lib):
    assert _reserve(lib, page=48) == NO and "page_size" in lib.attn_last_error().decode()
    assert _reserve(lib, B=0) == BAD
    assert _reserve(lib, T=-1) == BAD
    assert _reserve(lib, T=2**31 - 1) == BAD
    assert _reserve(lib, num_pages=0) == BAD
    assert _reserve(lib, num_pages=2**27) == NO
    assert _reserve(lib, blocks=0) == BAD
    assert _reserve(lib, blocks=2**28) == NO
    assert _reserve(lib, table=0x10002) == BAD and "aligned" in lib.attn_last_error().decode()
    assert _reserve(lib, table=None) == BAD and "NULL" in lib.attn_last_error().decode()
    # What is written is apart from everything else: sizes are 8, 2, 2, 9, 1 and 2, 3, 40, 40 numbers.
    for clash in (dict(lens=0x20004), dict(lens=0x30000), dict(cu=0x1001c), dict(slots=0x40000 - 39 * 4),
                  dict(positions=0x50000), dict(slots=0x90000), dict(pages=0x1001c), dict(free=0x20004),
                  dict(held=0x40020), dict(wanted=0x10000)):
        assert _reserve(lib, **clash) == BAD and "overlap" in lib.attn_last_error().decode(), clash
    for apart in (dict(lens=0x20008), dict(slots=0x40000 - 160), dict(held=0x30004), dict(T=0, slots=0x90000)):
        assert _reserve(lib, **apart) == BAD and "overlap" not in lib.attn_last_error().decode(), apart


def _shared(lib, *, q=16, strides=(512, 512, 64), table=16, prefix_blocks=5, length=16, lens=16, B=2, n_q=1, H=8, Hkv=2,
            d=64, pages=9, page=16, blocks=4, scale=0.125, ws=256, ws_bytes=1 << 40):
    return lib.attn_decode_shared_int8(q, *strides, 16, 16, 16, 16, table, prefix_blocks, length, 16, lens, 16, 16, B, n_q,
                                       H, Hkv, d, pages, page, blocks, F(scale), ws, ws_bytes, None)


def test_shared_arguments(lib):
    assert _shared(lib, page=48) == NO
    assert _shared(lib, d=96) == NO
    assert _shared(lib, H=9) == BAD
    assert _shared(lib, H=130) == NO
    assert _shared(lib, B=0) == BAD
    assert _shared(lib, n_q=0) == BAD
    assert _shared(lib, n_q=257) == NO
    assert _shared(lib, blocks=0) == BAD
    assert _shared(lib, prefix_blocks=0) == BAD and "prefix_blocks" in lib.attn_last_error().decode()
    assert _shared(lib, prefix_blocks=2**28) == NO
    assert _shared(lib, pages=2**27) == NO
    assert _shared(lib, scale=float("nan")) == BAD
    assert _shared(lib, scale=-1.0) == BAD
    assert _shared(lib, strides=(512, 516, 64)) == BAD and "q_token_stride" in lib.attn_last_error().decode()
    assert _shared(lib, q=None) == BAD
    assert _shared(lib, q=24) == BAD
    assert _shared(lib, B=2**23, n_q=256, H=8) == BAD
    # A short prefix is read by sequence, without a workspace; 64 sequences behind 2^20 positions need the own part's means
    # and sums, and a part of 256 rows for every run and unit at least.
    assert lib.attn_decode_shared_int8_workspace_bytes(2, 1, 8, 2, 64, 16, 5, 4) == 0
    need = lib.attn_decode_shared_int8_workspace_bytes(64, 1, 8, 2, 64, 16, 2**16, 4)
    assert need >= 64 * 8 * 66 * 4 + 3 * 256 * 66 * 4
    assert _shared(lib, B=64, prefix_blocks=2**16, ws_bytes=need - 1) == BAD
    assert lib.attn_decode_shared_int8_workspace_bytes(2, 1, 8, 3, 64, 16, 5, 4) == 0
    assert lib.attn_decode_shared_int8_workspace_bytes(2, 1, 8, 2, 64, 16, 0, 4) == 0


def test_binding_checks_tensors():
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    cache = [torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 16, 64, dtype=torch.int8),
             torch.zeros(3, 2), torch.zeros(3, 2)]
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_decode_shared_int8(q, *cache, ints, ints[:1], ints[None], ints[:1])
    with pytest.raises(ValueError):
        attn.attn_cache_reserve(ints[None], ints[:1], ints[:1], ints, ints[:1], 16, 4)
    with pytest.raises(ValueError):
        attn.attn_cache_reserve(ints, ints, ints, ints, ints[:1], 16, 4)


def test_reference_reserve_on_a_hand_example():
    """Pages of 16: sequence 0 ends and gives back two pages, 1 grows from 10 to 40 (two more), 2 gets its first."""
    table, stack = [[7, 3, -1], [5, -1, -1], [-1, -1, -1]], [1, 2, 0, 0, 0, 0, 0, 0]
    lens, cu, slots, positions, free = ref.reserve(table, [20, 10, 0], [0, 40, 2], stack, 2, 16, 34, 8)
    assert (lens, cu, free) == ([0, 40, 2], [0, 0, 30, 32], 1)
    # The stack is 1 2 7 3; of the top three, sequence 1 takes 2 and 7, sequence 2 takes 3.
    assert table == [[-1, -1, -1], [5, 2, 7], [3, -1, -1]]
    assert slots == [5 * 16 + i for i in range(10, 16)] + [2 * 16 + i for i in range(16)] + [
        7 * 16 + i for i in range(8)] + [48, 49, -1, -1]
    assert positions == list(range(10, 40)) + [0, 1, -1, -1]
    back = ref.reserve(table, lens, [20, 10, 0], stack, free, 16, 20, 8)
    assert table == [[7, 3, -1], [5, -1, -1], [-1, -1, -1]] and stack[:2] == [1, 2] and back[4] == 2


def test_reference_reserve_serves_in_order():
    """Two pages: the first request takes one, the second needs two and is not served, nor is the third; one that
    needs no page is."""
    table, stack = [[-1, -1], [-1, -1], [4, -1], [2, -1]], [3, 1]
    lens, cu, slots, _, free = ref.reserve(table, [0, 0, 16, 3], [5, 20, 17, 6], stack, 2, 16, 29, 5)
    assert lens == [5, 0, 16, 6] and cu == [0, 5, 25, 26, 29] and free == 1
    assert table == [[1, -1], [-1, -1], [4, -1], [2, -1]]
    assert slots == [16 + i for i in range(5)] + [-1] * 21 + [35, 36, 37]
