"""Which kernels the sizes of the GPU tests choose (CPU): every tile of the FP8 product, with its reduction in one piece
and in several, is run by one of them, and the choice written anew in block_plan.py is the library's."""
import random

import pytest

import block_plan as bp
from mixture_experts_layer_router_amd import block as lb
from test_gpu_block_forms import GRADIENTS, PRODUCTS


def test_the_figures_of_the_source_are_read():
    assert [(f[0], f[1]) for f in bp.FORMS] == [(4, 4), (4, 3), (2, 2), (1, 1)]
    assert all(len(f[3]) == f[2] and min(f[3]) > 0 for f in bp.FORMS)


def test_pieces_are_the_librarys():
    """A workspace holds the pieces in fp32, or 256 bytes where there is one."""
    rng = random.Random(5)
    sizes = list(PRODUCTS)
    for _ in range(3000):
        sizes.append((int(2 ** rng.uniform(0, 14.5)), 8 * int(2 ** rng.uniform(0, 11.5)), int(2 ** rng.uniform(0, 14.5))))
    for M, N, K in sizes:
        pieces = bp.plan(M, N, K)[1]
        want = 256 if pieces == 1 else -(-pieces * M * N * 4 // 256) * 256
        assert lb.lc_moe_matmul_fp8_workspace_size(M, N, K) == want, (M, N, K)


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_products_choose_what_they_are_listed_for(M, N, K):
    form, pieces = bp.plan(M, N, K)
    assert (form, pieces > 1) == PRODUCTS[M, N, K]


def test_every_form_is_listed_in_one_piece_and_in_several():
    assert set(PRODUCTS.values()) == {(f, s) for f in range(len(bp.FORMS)) for s in (False, True)}
    odd = {(PRODUCTS[s], -(-s[2] // 128) % 2) for s in PRODUCTS if not PRODUCTS[s][1]}
    assert len(odd) == 2 * len(bp.FORMS), "an odd and an even number of stages in every form"


@pytest.mark.parametrize("T,k,n", GRADIENTS)
def test_gradients_choose_what_they_are_listed_for(T, k, n):
    dx, dw = bp.plan(T, k, n), bp.plan(n, k, T)
    one = dx[0] == dw[0] and dx[0] >= 2 and dx[1] == dw[1] == 1
    assert (dx[0], dw[0], one) == GRADIENTS[T, k, n]


def test_both_gradients_in_one_launch_are_listed_for_every_form_that_has_it():
    assert {v[0] for v in GRADIENTS.values() if v[2]} == {2, 3}
