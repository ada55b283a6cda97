"""The native side of the binding on the CPU: arguments that do not fit leave no error and no call behind, only None,
so that the checks in Python name what is wrong."""
import pytest
import torch

import moe_grouped_gemm_nt_amd._lib as lib

bf = torch.bfloat16
NAMES = {"dg_route_balance": 8, "dg_route_balance_backward": 10, "dg_bf16_fp4_gemv_nt": 6, "dg_bf16_int4_gemv_nt": 7,
         "dg_m_grouped_bf16_fp4_gemv_nt_topk": 8, "dg_m_grouped_bf16_int4_gemv_nt_topk": 9, "dg_grad_norm": 3,
         "dg_grad_clip": 5}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("fill", [None, 3, 1 << 80, 2.5, "text", [], [5], (None,), object(), torch.zeros(2, 2),
                                  torch.zeros(2, 2).to_sparse(), torch.zeros(3, 4, 5), torch.zeros(1, device="meta"),
                                  [torch.zeros(3)]], ids=lambda v: type(v).__name__)
def test_arguments_that_do_not_fit(name, fill):
    fn = getattr(lib._load_native(), name)
    for n in (0, 1, NAMES[name], NAMES[name] + 1):
        assert fn(*[fill] * n) is None


def test_initialisation_names_what_is_missing():
    native = lib._load_native()
    with pytest.raises(TypeError, match="addresses"):
        native.init({})
    with pytest.raises(ValueError, match="no address of dg_route_balance"):
        native.init({}, None, None)
