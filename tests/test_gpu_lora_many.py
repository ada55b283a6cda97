"""Adapters over more tokens than one grid has threads for, on a stream whose bound
workspace has room for them all: the tokens then still go through in parts."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_tokens_than_a_grid():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as dg
    T = 2 ** 30 + 70                    # 64 tokens to a workgroup of 256
    print(f"case: adapters over {T} tokens with a workspace of 10 GiB", flush=True)
    st = torch.cuda.Stream()
    z = dict(dtype=torch.bfloat16, device="cuda")
    c = torch.arange(T, dtype=torch.int32, device="cuda").remainder_(251).to(torch.bfloat16).view(T, 1)
    d = torch.full((T, 1), -1.0, **z)
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    x = torch.empty(1, **z).as_strided((T, 0), (8, 1))          # no adapters: nothing of x is read
    space = torch.empty(10 << 30, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    dg.dg_bind_stream_workspace(st, space)
    try:
        dg.dg_lora_bf16_nt(x, torch.empty(0, 16, 0, **z), torch.empty(0, 1, 16, **z), None, ids, c, d, stream=st)
        st.synchronize()
    finally:
        dg.dg_bind_stream_workspace(st, None)
    assert torch.equal(c, d)
    del c, d, ids, space
    torch.cuda.empty_cache()
