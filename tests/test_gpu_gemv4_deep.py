"""The 4-bit products on every launch shape with more pieces of K per wave than its LDS
holds at a time, an odd last half among them, and tiles of every fullness; to the bit
(tests/exact4.py)."""
import numpy as np
import pytest
import torch

from tests.exact4 import FORMS, decode, generator, of_expert, product, quarters, weights, whole
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_grouped_gemm_nt_amd as m
    yield m
    torch.cuda.empty_cache()


def dense(dg, form):
    return dg.dg_bf16_fp4_gemv_nt if form == "fp4" else dg.dg_bf16_int4_gemv_nt


def by_choice(dg, form):
    return dg.dg_m_grouped_bf16_fp4_gemv_nt_topk if form == "fp4" else dg.dg_m_grouped_bf16_int4_gemv_nt_topk


def same(d, want, what):
    bad = (d != want).nonzero()
    assert not len(bad), (what, len(bad), bad[:3].tolist(), d[tuple(bad[0])], want[tuple(bad[0])])


# At 256 CUs: columns per workgroup 64, 64 (32 for groups of 32), 32 and 16 in tiles of 16 tokens, of which the last has
# 1, 3, 6 or 12; 32, 32 and 16 in tiles of 8 and of 4.  65 pieces of 256 K are 8 or more per wave, 33 as many for four
# waves, 16 (with which tiles of 4 have a shape of their own) four.
LARGE, MIDDLE, SMALL = 16512, 8320, 3968
SIZES = [
    (49, 4200, MIDDLE), (51, 4200, MIDDLE), (54, 4200, MIDDLE), (60, 4200, LARGE),
    (49, 2112, LARGE), (51, 2112, LARGE), (54, 2112, LARGE), (64, 2112, LARGE),
    (17, 2112, LARGE), (19, 2112, LARGE), (22, 2112, MIDDLE), (28, 2112, LARGE),
    (9, 100, LARGE), (17, 100, LARGE), (19, 100, LARGE), (22, 100, LARGE), (32, 100, 16384),
    (8, 8300, MIDDLE), (5, 8300, LARGE), (7, 4200, LARGE), (6, 500, LARGE),
    (1, 8300, LARGE), (3, 8300, MIDDLE), (1, 8300, SMALL), (4, 8300, SMALL), (2, 4200, LARGE), (4, 4200, LARGE),
    (1, 77, LARGE), (4, 77, LARGE),
]


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_dense(dg, size, form):
    M, N, K = size
    print(f"case: exact gemv {size} {form}", flush=True)
    g = generator(M + N + K)
    args, x, c = weights(g, form, (), N, K), whole(g, M, K), quarters(g, M, N)
    want = product(x, decode(form, *args), c)
    d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dense(dg, form)(x, *args, c, d)
    torch.cuda.synchronize()
    same(d, want, (size, form))


# token by token which experts it takes, so that they have the given numbers of choices; the columns after each other make
# 64, 64 (32), 32 and 16 columns per workgroup of the tiles that there can be
def one_each(counts, T):
    """ids [T][1]: counts[e] tokens of expert e, the others of none that is here, in turn"""
    ids = np.concatenate([np.full(n, e) for e, n in enumerate(counts)] + [np.full(T - sum(counts), -1)])
    return ids[np.random.default_rng(T).permutation(T)].astype(np.int32).reshape(T, 1)


def side_by_side(T, *columns):
    """ids [T][len(columns)]: each column's experts from the first token on, then none"""
    ids = np.full((T, len(columns)), -1, dtype=np.int32)
    for j, column in enumerate(columns):
        ids[:len(column), j] = column
    return ids


SIXTEEN = one_each([1, 3, 6, 12, 16, 20], 60)
EIGHT = side_by_side(8, [3] * 8, [2] * 6, [1] * 3 + [0])
FOUR = side_by_side(4, [3] * 4, [0, 1, 1, 9], [2] * 3)
CHOICES = [
    (SIXTEEN, 1650, MIDDLE), (SIXTEEN, 820, LARGE), (SIXTEEN, 410, LARGE), (SIXTEEN, 90, LARGE),
    (EIGHT, 1060, MIDDLE), (EIGHT, 530, LARGE), (EIGHT, 90, LARGE),
    (FOUR, 1190, MIDDLE), (FOUR, 1190, SMALL), (FOUR, 590, LARGE), (FOUR, 90, LARGE),
    (one_each([300, 1, 17, 500, 0, 31, 200], 1100), 70, 4224), (one_each([7] * 150, 1056), 40, 2176),
]


@pytest.mark.parametrize("per_choice", [False, True])
@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("case", range(len(CHOICES)), ids=lambda i: f"{CHOICES[i][0].shape}x{CHOICES[i][1]}x{CHOICES[i][2]}")
def test_by_choice(dg, case, form, per_choice):
    ids, N, K = CHOICES[case]
    T, k = ids.shape
    G = int(ids.max()) + 1 if ids.max() < 9 or T > 100 else 4
    print(f"case: exact gemv by choice {ids.shape} of {G}, {N}x{K} {form} {per_choice}", flush=True)
    check_choices(dg, form, ids, G, N, K, per_choice, generator(T + N + K))


def check_choices(dg, form, ids, G, N, K, per_choice, g, first=0):
    T, k = ids.shape
    args = weights(g, form, (G,), N, K)
    x, c = whole(g, T * k if per_choice else T, K), quarters(g, T * k, N)
    d = c.clone()
    by_choice(dg, form)(x, dev(ids + np.int32(first)), first, *args, d, d)
    torch.cuda.synchronize()
    flat = torch.from_numpy(ids.ravel()).cuda()
    rows = x if per_choice else x.repeat_interleave(k, 0)
    want = c.clone()
    for e in range(G):
        at = (flat == e).nonzero().view(-1)
        if len(at):
            want[at] = product(rows[at], decode(form, *of_expert(args, e)), c[at])
    same(d, want, (ids.shape, G, N, K, form))


@pytest.mark.parametrize("form", FORMS[1:], ids=str)
def test_integers_with_the_largest_x(dg, form):
    """x up to 2^116 and scales as small: a group's sums reach 2^127, the results are those of the small numbers."""
    g = generator(1)
    M, N, K = 9, 40, 1152
    b, s, z = weights(g, form, (), N, K)
    x, c = whole(g, M, K), quarters(g, M, N)
    x[3], x[4] = 2.0, -2.0                       # sums of one sign
    want = product(x, decode(form, b, s, z), c)
    d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dense(dg, form)(x * 2.0 ** 115, b, s * 2.0 ** -115, z, c, d)
    torch.cuda.synchronize()
    same(d, want, form)
