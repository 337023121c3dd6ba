"""Which tile a product of microscaled operands runs on, asked of the library's own plan (no
GPU): the shapes that test_gpu_mx_tiles.py takes for each tile do run on it, in every kind, so
that a change to the plan cannot take a tile out of the tests unnoticed."""
import pytest
import torch

from layer_wise_obs_amd import _lib as L

BF, F32 = torch.bfloat16, torch.float32
KINDS = [(form, ydt) for form in ("e4m3", "e2m1") for ydt in (BF, F32)]
# tile (tokens, channels): tokens and channels of products that run on it whole, with any
# contraction of WHOLE_K; none is a multiple of its tile
WHOLE = {(16, 16): (15, 333), (64, 64): (300, 263), (128, 128): (1003, 2101), (128, 256): (19055, 157),
         (256, 256): (9747, 795)}
WHOLE_K = [96, 288, 640, 1056]
JOINED = [(70, 4096, 521), (100, 4096, 15), (301, 4096, 263)]  # contractions in pieces
PAST_CACHE = (131101, 96, 1031)  # 2^27 outputs and more


@pytest.mark.parametrize("tile", WHOLE)
@pytest.mark.parametrize("b", WHOLE_K)
def test_shapes_run_on_their_tile(tile, b):
    n, c = WHOLE[tile]
    for form, ydt in KINDS:
        assert L.debug_mx_linear_plan(form, n, b, c, ydt) == (*tile, 1), (form, ydt)


@pytest.mark.parametrize("n,b,c", JOINED)
def test_shapes_run_in_pieces(n, b, c):
    for form, ydt in KINDS:
        assert L.debug_mx_linear_plan(form, n, b, c, ydt)[2] > 1
        assert L.debug_mx_linear_plan(form, n, b, c, ydt, ws=False)[2] == 1
        assert L.mx_linear_workspace_size(form, n, b, c, ydt) > 0


def test_largest_outputs_run_on_the_largest_tile():
    n, b, c = PAST_CACHE
    assert n * c >= 2 ** 27
    assert L.debug_mx_linear_plan("e4m3", n, b, c, BF) == (256, 256, 1)


def test_plan_refuses_what_the_product_refuses():
    for args in (("e4m3", 8, 40, 8), ("e4m3", -1, 64, 8), ("e2m1", 8, 64, 0), ("e2m1", 0, 64, 8)):
        with pytest.raises(L.ThanosError):
            L.debug_mx_linear_plan(*args, BF)
