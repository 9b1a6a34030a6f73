"""Serving entry points: host-side checks at the ends of their ranges (no kernel is launched)."""
import ctypes

import pytest

from precision_numerics_gb300 import attn, build

F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


def test_numbers_of_sequences_that_a_stride_would_pass(lib):
    """The kernels go over the sequences in strides of up to 1024 in 32 bits."""
    for B in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 1024):
        calls = (
            lambda: lib.attn_varlen_plan(16, B, 3, 1, 1, 1, 16, 1 << 50, None),
            lambda: lib.attn_varlen_fwd(16, 16, 16, 64, 64, 64, 64, 64, 64, 16, 1 << 50, 16, 16, B, 3, 1, 1, 64, F(0.1), 1,
                                        None),
            lambda: lib.attn_cache_append_int8(16, 16, 64, 64, 64, 64, 16, 16, 16, 16, 16, 16, 16, B, 3, 1, 64, 9, 16, 4,
                                               None),
            lambda: lib.attn_cache_read_int8(16, 16, 16, 16, 16, 16, 16, 16, 16, B, 3, 1, 64, 9, 16, 4, 1, None),
            lambda: lib.attn_decode_int8(16, 64, 64, 64, 16, 16, 16, 16, 16, 16, 16, 16, B, 1, 1, 1, 64, 9, 16, 4, F(0.1),
                                         256, 1 << 50, None),
        )
        for call in calls:
            assert call() == attn.ATTN_ERR_INVALID_ARG
            assert "too large" in lib.attn_last_error().decode()
        assert lib.attn_varlen_plan_bytes(B, 3, 1, 1) == 0
        assert lib.attn_decode_int8_workspace_bytes(B, 1, 1, 1, 64, 16, 4) == 0


def test_workspace_of_invalid_arguments_is_zero(lib):
    """What attn_decode_int8 refuses needs no workspace."""
    good = dict(B=2, n_q=1, H=8, Hkv=2, d=64, page=16, blocks=4000)

    def need(**kw):
        x = {**good, **kw}
        return lib.attn_decode_int8_workspace_bytes(x["B"], x["n_q"], x["H"], x["Hkv"], x["d"], x["page"], x["blocks"])

    assert need() > 0
    for kw in (dict(page=17), dict(page=256), dict(page=-16), dict(blocks=0), dict(blocks=-1), dict(blocks=2 ** 28),
               dict(d=96), dict(H=9), dict(n_q=257), dict(B=0)):
        assert need(**kw) == 0, kw


def test_plan_has_room_for_items_of_one_tile(lib):
    """An item is 128 // G tokens of a sequence where pairs of tiles would not fill the SMs: the plan's
    16-byte entries behind its header suffice for every way to cut T tokens into B sequences."""
    for H, Hkv in ((1, 1), (8, 2), (6, 2), (64, 1), (5, 1)):
        tq = 128 // (H // Hkv)
        for B in (1, 2, 5):
            for T in (0, 1, tq - 1, tq, tq + 1, 2 * tq + 1, 7 * tq + 3):
                cuts = [[T] + [0] * (B - 1)]
                for x in (1, tq - 1, tq, tq + 1, 2 * tq + 1):  # B - 1 sequences of x tokens, as far as there are any
                    cut = [max(0, min(x, T - x * i)) for i in range(B - 1)]
                    cuts.append(cut + [T - sum(cut)])
                items = max(sum(-(-n // tq) for n in cut) for cut in cuts)
                assert items <= (lib.attn_varlen_plan_bytes(B, T, H, Hkv) - 256) // 16
