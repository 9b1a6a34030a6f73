"""Serving entry points: host-side checks (no kernel is launched), and the plain forms the GPU
tests compare with."""
import ctypes

import pytest
import torch

import serving_ref as ref
from precision_numerics_gb300 import attn, build

F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


def _prompt(lib, *, q=16, k=16, strides=(512, 64, 128, 64, 128, 64), plan=16, plan_bytes=1 << 20, B=2, T=40,
            H=8, Hkv=2, d=64, scale=0.125):
    return lib.attn_varlen_fwd(q, k, 16, *strides, plan, plan_bytes, 16, 16, B, T, H, Hkv, d, F(scale), 1, None)


def test_prompt_arguments(lib):
    bad, no = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    assert _prompt(lib, d=96) == no
    assert _prompt(lib, H=7) == bad and "multiple" in lib.attn_last_error().decode()
    assert _prompt(lib, H=130, Hkv=2) == no
    assert _prompt(lib, B=0) == bad
    assert _prompt(lib, T=-1) == bad
    assert _prompt(lib, scale=float("inf")) == bad
    assert _prompt(lib, scale=0.0) == bad
    assert _prompt(lib, strides=(516, 64, 128, 64, 128, 64)) == bad
    assert "q_token_stride" in lib.attn_last_error().decode()
    assert _prompt(lib, strides=(512, 64, 128, 64, 128, -64)) == bad
    assert _prompt(lib, plan_bytes=256) == bad and "plan" in lib.attn_last_error().decode()
    assert _prompt(lib, q=None) == bad and "NULL" in lib.attn_last_error().decode()
    assert _prompt(lib, q=24) == bad and "aligned" in lib.attn_last_error().decode()
    assert _prompt(lib, T=2**31 - 1, B=2**30, Hkv=8, H=8) == bad
    assert _prompt(lib, T=0, q=None) == attn.ATTN_OK  # nothing to do, nothing is launched


def test_plan_bytes_cover_every_split_of_the_tokens(lib):
    """Items of 2 * (128 // G) tokens: every way to cut T tokens into B sequences fits the plan."""
    for H, Hkv in ((1, 1), (8, 2), (6, 2), (64, 1), (5, 1)):
        per = 2 * (128 // (H // Hkv))
        for B in (1, 2, 5):
            for T in (0, 1, per - 1, per, per + 1, 3 * per + 7):
                room = (lib.attn_varlen_plan_bytes(B, T, H, Hkv) - 256) // 16
                worst = max(sum(-(-n // per) for n in cut) for cut in _cuts(T, B, per))
                assert worst <= room
    assert lib.attn_varlen_plan_bytes(0, 5, 1, 1) == 0
    assert lib.attn_varlen_plan(16, 2, 40, 8, 2, 1, 16, 100, None) == attn.ATTN_ERR_INVALID_ARG
    assert lib.attn_varlen_plan(None, 2, 40, 8, 2, 1, 16, 1 << 20, None) == attn.ATTN_ERR_INVALID_ARG
    assert lib.attn_varlen_plan(18, 2, 40, 8, 2, 1, 16, 1 << 20, None) == attn.ATTN_ERR_INVALID_ARG


def _cuts(T, B, per):
    yield [T] + [0] * (B - 1)
    ones = [min(1, max(0, T - i)) for i in range(B - 1)]
    yield ones + [T - sum(ones)]
    for x in (per - 1, per, per + 1):
        if x * (B - 1) <= T:
            yield [x] * (B - 1) + [T - x * (B - 1)]


def _append(lib, *, k=16, strides=(128, 64, 128, 64), cache=16, scale=16, table=16, cu=16, starts=16, B=2, T=3,
            Hkv=2, d=64, pages=9, page=16, blocks=4):
    return lib.attn_cache_append_int8(k, 16, *strides, cache, 16, scale, 16, table, cu, starts, B, T, Hkv, d, pages,
                                      page, blocks, None)


def _read(lib, *, dt=1, page=16, d=64, out=16, T=3, blocks=4):
    return lib.attn_cache_read_int8(16, 16, 16, 16, 16, 16, 16, out, 16, 2, T, 2, d, 9, page, blocks, dt, None)


def _decode(lib, *, q=16, strides=(512, 512, 64), lens=16, B=2, n_q=1, H=8, Hkv=2, d=64, pages=9, page=16, blocks=4,
            scale=0.125, ws=256, ws_bytes=1 << 30):
    return lib.attn_decode_int8(q, *strides, 16, 16, 16, 16, 16, lens, 16, 16, B, n_q, H, Hkv, d, pages, page, blocks,
                                F(scale), ws, ws_bytes, None)


def test_cache_arguments(lib):
    bad, no = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    for call in (_append, _read, _decode):
        assert call(lib, page=48) == no and "page_size" in lib.attn_last_error().decode()
        assert call(lib, page=256) == no
        assert call(lib, d=32) == no
        assert call(lib, blocks=0) == bad
    assert _append(lib, pages=0) == bad
    assert _append(lib, pages=2**27, page=128) == no
    assert _append(lib, B=0) == bad
    assert _append(lib, T=-1) == bad
    assert _append(lib, strides=(128, 63, 128, 64)) == bad
    assert _append(lib, cache=None) == bad
    assert _append(lib, cache=8) == bad
    assert _append(lib, scale=18) == bad
    assert _append(lib, table=None) == bad
    assert _append(lib, cu=17) == bad
    assert _read(lib, dt=5) == bad
    assert _read(lib, out=None) == bad
    assert _decode(lib, n_q=0) == bad
    assert _decode(lib, n_q=257) == no
    assert _decode(lib, H=9) == bad
    assert _decode(lib, scale=float("nan")) == bad
    assert _decode(lib, strides=(512, 512, 60)) == bad
    assert _decode(lib, q=None) == bad
    assert _decode(lib, lens=19) == bad
    assert _decode(lib, blocks=2**28) == no
    assert lib.attn_decode_int8_workspace_bytes(0, 1, 8, 2, 64, 16, 4) == 0


def test_binding_checks_tensors():
    """Shapes, types and devices are refused before the library is called."""
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn.attn_varlen_fwd(q, q, q, torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError):
        attn.attn_varlen_plan(torch.zeros(3, dtype=torch.int32), 4, 2, 2)
    cache = [torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 16, 64, dtype=torch.int8),
             torch.zeros(3, 2), torch.zeros(3, 2), torch.zeros(1, 2, dtype=torch.int32)]
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_cache_append_int8(q, q, *cache, ints, ints[:1])
    with pytest.raises(ValueError):
        attn.attn_cache_read_int8(*cache, ints, ints[:1], 4)
    with pytest.raises(ValueError):
        attn.attn_decode_int8(q[None], *cache, ints[:1])


def test_reference_attention_on_a_hand_example():
    """Two keys with scores ln 1 and ln 3: p = 1/4, 3/4."""
    q = torch.tensor([[1.0, 0.0]])
    k = torch.tensor([[0.0, 5.0], [3.0, 0.0]]).double()
    k[1, 0] = torch.log(torch.tensor(3.0, dtype=torch.float64))
    v = torch.tensor([[4.0, 0.0], [0.0, -8.0]])
    o, lse, a, size = ref.attention(q, k, v, 1.0, [1])
    assert torch.allclose(o, torch.tensor([[1.0, -6.0]], dtype=torch.float64))
    assert torch.allclose(lse, torch.log(torch.tensor([4.0], dtype=torch.float64)))
    assert torch.allclose(a, torch.tensor([[1.0, 6.0]], dtype=torch.float64))
    o, lse, _, _ = ref.attention(q, k, v, 1.0, [-1])
    assert torch.equal(o, torch.zeros(1, 2, dtype=torch.float64)) and lse[0] == -torch.inf


def test_reference_append_on_a_hand_example():
    """Fresh page: a = 254, s = 2, 127 lies on the border between 63 and 64 (even: 64).  A larger
    value later doubles the scale and halves the codes, ties to even."""
    codes = torch.full((1, 1, 16, 64), 9, dtype=torch.int8)
    scales = torch.full((1, 1), 5.0)
    rows = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    rows[0, 0, :4] = torch.tensor([254.0, 127.0, -126.0, 3.0])
    ref.append(rows, codes, scales, [0], 0)
    assert scales[0, 0] == 2.0
    assert codes[0, 0, 0, :5].tolist() == [127, 64, -63, 2, 0] and codes[0, 0, 2, 0] == 9
    rows = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    rows[0, 0, :2] = torch.tensor([508.0, torch.inf])
    ref.append(rows, codes, scales, [0], 2)
    assert scales[0, 0] == 4.0
    assert codes[0, 0, 0, :4].tolist() == [64, 32, -32, 1] and codes[0, 0, 2, :2].tolist() == [127, 127]
