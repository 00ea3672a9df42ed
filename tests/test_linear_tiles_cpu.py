"""Which tiles the linear layers' shapes take: what the GPU tests of the tiles rely on."""
import ctypes

import pytest

import routing_expert_ffn_router_amd as moe
from _linear_tiles import CASES, SCAN, pieces_of, shape_of


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}-{c[3]}-E{len(c[4])}")
def test_the_case_takes_the_tiles_it_is_for(case):
    assert moe.linear_tiles(shape_of(case))[:2] == (case[1], case[2])
    assert (pieces_of(case) > 1) == case[3]


def test_every_form_is_there_whole_and_cut_with_and_without_a_table():
    seen = {(c[0], c[1], c[2], c[3], len(c[4]) > SCAN) for c in CASES}
    for form in (("bf16", 64, 256), ("bf16", 128, 256), ("bf16", 256, 256), ("f32", 128, 256)):
        for cut in (False, True):
            for table in (False, True):
                assert (*form, cut, table) in seen
    # rows that end inside either band of a tile, and inside 16 rows
    for form in {c[:3] for c in CASES}:
        rest = {n % form[1] for c in CASES if c[:3] == form for n in c[4] if n % 16}
        assert any(0 < r < form[1] // 2 for r in rest) and any(r > form[1] // 2 for r in rest)


def test_refusals():
    with pytest.raises(moe.MoeError):
        moe.linear_tiles(moe.group_shape(10, 1, 100, 128))
    lib = moe.load_library()
    g = moe.group_shape(10, 1, 128, 128)
    assert lib.moe_linear_tiles(ctypes.byref(g), None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_tiles(None, (ctypes.c_int64 * 3)()) == moe.MOE_ERR_INVALID_ARG
    assert moe.linear_tiles(moe.group_shape(0, 1, 128, 128))[2] == 1
