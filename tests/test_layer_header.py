"""What include/dg.h says of roundings and ranges in the balance loss, the 4-bit products and the clipping."""
import pytest

from tests.test_layer_refusals import comment_of


@pytest.mark.parametrize("name,said", [
    ("dg_route_balance", "(E + 160 + T / 4096) * 2^-24 of itself"),
    ("dg_bf16_int4_gemv_nt", "the sums do where x is below 2^117 in magnitude"),
    ("dg_bf16_fp4_gemv_nt", "in tiles of 4, 8 or 16 tokens"),
    ("dg_m_grouped_bf16_fp4_gemv_nt_topk", "4, 8 or 16 at a time"),
    ("dg_grad_clip", "those of bf16 tensors rounded once more to bf16"),
])
def test_said(name, said):
    assert said in comment_of(name)


def test_the_largest_x_whose_sums_stay_in_range():
    """15 * 128 values of 2^117 less one step of bf16 are below fp32's largest value, of 2^118 beyond."""
    most = (2.0 - 2.0 ** -23) * 2.0 ** 127
    assert 15 * 128 * 2.0 ** 117 * (1 - 2.0 ** -9) < most < 15 * 128 * 2.0 ** 118
