"""CPU: token counts whose product with top_k or H passes 64 bits are refused like any other
count past the limits (nothing reaches a GPU)."""

import os

import pytest

from w4a16_group_quantized_amd import ops

FAKE = 0x1000  # aligned and never dereferenced: validation fails first
WRAPS = [1 << 62, (1 << 62) + 1, 1 << 60, (1 << 63) - 1, (1 << 32) + 1, 1 << 31]  # of T x 4 and T x 64


@pytest.fixture(scope="module", autouse=True)
def _built_library():
    if not os.path.exists(ops.LIB_PATH):
        from w4a16_group_quantized_amd import build_lib

        build_lib.build()


def _calls(lib, T):
    k, E, H, I, P, big = 4, 8, 64, 32, FAKE, 1 << 62
    yield "moe_permute_masked", (P, T, k, 0, E, P, P, P, P, P, P, big, None)
    yield "moe_dispatch", (P, 1, T, k, H, H, P, 16, P, H, None)
    yield "moe_dispatch_backward", (P, 1, T, k, H, H, P, 16, P, H, None)
    yield "moe_combine_masked", (P, 1, T, k, H, H, P, P, 16, P, 1, H, None)
    yield "moe_combine_backward", (P, 1, H, P, 1, H, P, P, T, k, H, 16, P, H, P, None)
    yield "moe_mxfp4_layer_forward", (P, P, 1, T, E, k, P, P, P, P, H, I, P, P, big, None)
    yield "moe_mxfp4_quantize", (P, 1, T, H, H, P, P, None)
    yield "moe_mxfp4_grouped_gemm", (P, P, T, P, k, 16, P, E, P, P, H, H, P, 1, H, None)
    yield "moe_route", (P, T, E, k, P, P, None)
    yield "moe_router_gate", (P, T, H, P, E, P, None)
    yield "moe_permute", (P, T, k, E, P, P, P, P, P, P, big, None)
    yield "moe_combine", (P, P, P, T, k, H, P, None)


@pytest.mark.parametrize("T", WRAPS)
def test_token_counts_past_the_limits_are_refused(T):
    lib = ops.load_library()
    for name, args in _calls(lib, T):
        assert getattr(lib, name)(*args) == ops.MOE_ERR_UNSUPPORTED, (name, T)
    assert ops.permute_masked_workspace_bytes(T, 4, 8) == 0
    assert ops.mxfp4_layer_workspace_bytes(T, 4, 8, 64, 32) == 0
