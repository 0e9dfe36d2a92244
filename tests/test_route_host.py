"""Routing by scores: refusals that need no GPU, of outputs that are inputs."""

import ctypes

import pytest

import fp8_block_scale_amd as moe

LOGITS, BIAS, IDS, WEIGHTS = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(4))      # never dereferenced


def _route(M=4, logits=LOGITS, bias=BIAS, ids=IDS, weights=WEIGHTS):
    return moe.STATUS_NAMES[moe._c["moe_route_scored"](logits, moe.MOE_DT_F32, M, 16, 16, 2, moe.MOE_SCORE_SIGMOID,
                                                       bias, 4, 2, 2, 1, 1.0, 1, ids, weights, None)]


@pytest.mark.parametrize("bias", [BIAS, None])
def test_an_output_that_is_an_input(bias):
    """The weights are computed from logits read after the ids are written."""
    assert _route(bias=bias, ids=LOGITS) == "MOE_ERR_SHAPE"
    assert _route(bias=bias, weights=LOGITS) == "MOE_ERR_SHAPE"
    assert _route(bias=bias, weights=IDS) == "MOE_ERR_SHAPE"
    if bias:
        assert _route(ids=bias) == "MOE_ERR_SHAPE"
        assert _route(weights=bias) == "MOE_ERR_SHAPE"


def test_nothing_to_do_needs_no_tensors():
    assert _route(M=0, logits=None, bias=None, ids=None, weights=None) == "MOE_OK"
