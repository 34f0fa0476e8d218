"""Serving C ABI without a GPU: sizes past the 32-bit indices of the kernels are
refused before any launch."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
from test_serve_abi import I31, INVALID, attn, lib, no_gpu, plan  # noqa: F401

MOST = 1 << 30


@no_gpu
def test_requests_past_the_limit_are_refused(lib):  # noqa: F811
    for B in (MOST + 1, I31 - 255, I31):
        assert plan(lib, B=B, width=1, wsz=1 << 36) == INVALID, B
        assert attn(lib, B=B, width=1, wsz=1 << 36) == INVALID, B


@pytest.mark.parametrize("B", [MOST + 1, I31 - 255, I31])
def test_workspace_queries_refuse_them(B):
    assert kda.kda_page_plan_workspace_size(B) == 0
    assert kda.kda_attn_paged_workspace_size(8, B, 8, 2, 64, 0, torch.bfloat16) == 0


def test_the_limit_itself_has_a_workspace():
    assert kda.kda_page_plan_workspace_size(MOST) > 0
    assert kda.kda_attn_paged_workspace_size(8, MOST, 8, 2, 64, 0, torch.bfloat16) > 0


@no_gpu
def test_scales_whose_product_with_log2_e_overflows_are_refused(lib):  # noqa: F811
    for scale in (1.01 * 2.0 ** 127, 2.5e38, 3.4028234e38):
        assert attn(lib, scale=scale) == INVALID, scale
    for scale in (0.0, 1.0, 2.0 ** 127):
        assert attn(lib, scale=scale) != INVALID, scale
