"""Every ring of stages that the layer for a few tokens may take, against the 64-bit form: by the number
of tokens, in one and in two pieces of 128 bytes a step, and with as many experts as there may be, whose
tables leave the ring less room."""
import pytest
import torch

from test_gpu_few import KINDS, _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", range(1, 17))
def test_two_pieces_a_step(T, kind):
    c = _case(T, 6, 2, 512, 768, kind, seed=100 + T)
    _check(c, *_run(c))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", range(1, 17))
def test_one_piece_a_step(T, kind):  # (in 8 bits; wider rows are whole pairs of pieces)
    c = _case(T, 5, 2, 384, 640, kind, seed=200 + T)
    _check(c, *_run(c))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,k", [(1, 1024, 8), (5, 640, 16), (8, 480, 8), (8, 1024, 64), (9, 1024, 16),
                                   (13, 600, 8), (16, 1024, 32)])
def test_many_experts(T, E, k, kind):
    c = _case(T, E, k, 128, 128, kind, seed=E + k)
    out, ints = _run(c)
    _check(c, out, ints)
    assert int(ints[0].sum()) == T * k


@pytest.mark.parametrize("kind", ["e4m3-f32", "e4m3-e8m0"])
@pytest.mark.parametrize("T,d,F", [(9, 2048, 1024), (13, 1024, 2048), (8, 2048, 1024), (16, 1024, 1024)])
def test_rings_that_go_round(T, d, F, kind):
    """Reductions of more steps than the ring has stages, down's in chunks."""
    c = _case(T, 4, 2, d, F, kind, seed=d + T)
    out, ints = _run(c)
    _check(c, out, ints)
    assert torch.equal(out, _run(c, ws_byte=0)[0])
