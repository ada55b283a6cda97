"""The 4-bit products that go out in several launches (lists that do not fit, more
workgroups than a launch has) and the longest K; to the bit (tests/exact4.py)."""
import numpy as np
import pytest
import torch

from tests.exact4 import FORMS, decode, draw, generator, of_expert, product, weights, whole
from tests.test_gpu_gemv4_deep import check_choices, dense, same
from tests.workspaces import Bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    yield m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form", [FORMS[0], FORMS[3]], ids=str)
@pytest.mark.parametrize("n,room,per_choice", [
    (7001, 26 * 1024, False), (7001, 26 * 1024, True),           # lists of 1750, 2625 and 2626 choices
    (4000, 17 * 1024 + 512, True),                               # twice 2000
    (9000, 65536, False),                                        # 4500 twice
    (20011, 81408, True),                                        # 10005 and 10006, with room for the lists only
    (1900, 1024, False),                                         # 1024 and 876 without lists
])
def test_lists_in_several_launches(dg, n, room, per_choice, form):
    print(f"case: gemv of {n} choices with {room} bytes for lists, {form} {per_choice}", flush=True)
    rng = np.random.default_rng(n + room)
    k = 1 if n % 2 else 2
    ids = rng.integers(-1, 8, (n // k, k)).astype(np.int32)
    with Bound(dg, room):
        check_choices(dg, form, ids, 7, 40, 640, per_choice, generator(n + 1), first=5)


def test_more_columns_than_one_launch(dg):
    """300 tiles of 2^20 columns, 64 to a workgroup: the columns go out in two launches."""
    print("case: gemv 4800 x 2^20", flush=True)
    M, N, K = 4800, 1 << 20, 128
    g = generator(0)
    args, x = weights(g, "fp4", (), N, K), whole(g, M, K)
    d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_fp4_gemv_nt(x, *args, None, d)
    torch.cuda.synchronize()
    for n in range(0, N, 1 << 16):
        at = slice(n, n + (1 << 16))
        w = decode("fp4", args[0][at], args[1][:, at].contiguous())
        assert torch.equal(d[:, at], (x.float() @ w.float().t()).to(torch.bfloat16)), n


def test_more_tiles_than_one_launch(dg):
    """Beyond 2^26 tokens the tiles go out in two launches."""
    print("case: gemv of 2^26 + 37 tokens", flush=True)
    M, N, K = (1 << 26) + 37, 3, 128
    g = generator(1)
    args = weights(g, "fp4", (), N, K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    step = 1 << 22
    for at in range(0, M, step):
        part = x[at:at + step]
        part.copy_(draw(g, -2, 3, *part.shape, dtype=torch.int8))
    d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_fp4_gemv_nt(x, *args, None, d)
    torch.cuda.synchronize()
    w = decode("fp4", *args).float().t().contiguous()
    for at in range(0, M, step):
        assert torch.equal(d[at:at + step], (x[at:at + step].float() @ w).to(torch.bfloat16)), at


def test_more_tiles_of_choices_than_one_launch(dg):
    """68 million choices, listed in 0.6 GB, in two launches."""
    print("case: gemv of 68 million choices", flush=True)
    T, k, G, N, K = 1100007, 62, 3, 1, 128
    g = generator(3)
    args, x, ids = weights(g, "fp4", (G,), N, K), whole(g, T, K), draw(g, -1, G + 1, T, k, dtype=torch.int32)
    d = torch.full((T * k, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    with Bound(dg, 1 << 30):
        dg.dg_m_grouped_bf16_fp4_gemv_nt_topk(x, ids, 0, *args, None, d)
    y = torch.stack([(x.float() @ decode("fp4", *of_expert(args, e)).float().t()).view(T) for e in range(G)], 1)
    y = torch.cat([y, torch.zeros(T, 2, device="cuda")], 1).to(torch.bfloat16)
    want = y.gather(1, torch.where(ids < 0, torch.full_like(ids, G), ids).long())
    assert torch.equal(d.view(T, k), want)


@pytest.mark.parametrize("form", ["fp4", ("int4", 128, "float32", True)], ids=str)
def test_the_longest_k(dg, form):
    """K of 2^24, of which x has 156 blocks of 128 that are not zero: sums as of K = 20000."""
    print(f"case: gemv of K = 2^24 {form}", flush=True)
    N, K = 130, 1 << 24
    g = generator(6)
    args = [t for t in weights(g, form, (), N, K)]
    for M in (1, 3):
        blocks = torch.randperm(K // 128, device="cuda", generator=g)[:156].sort().values
        blocks[0], blocks[-1] = 0, K // 128 - 1
        x = torch.zeros(M, K // 128, 128, dtype=torch.bfloat16, device="cuda")
        x[:, blocks] = whole(g, M, len(blocks), 128)
        d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        dense(dg, form)(x.view(M, K), *args, None, d)
        torch.cuda.synchronize()
        here = [args[0].view(N, K // 128, 64)[:, blocks].reshape(N, -1)] + [t[blocks].contiguous() for t in args[1:]]
        same(d, product(x[:, blocks].reshape(M, -1), decode(form, *here)), (form, M))
