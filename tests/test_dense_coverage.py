"""CPU: the linear layer's test sizes reach every body that the choosing rules can choose, whole and in pieces."""
import pytest

import dense_cases as cases
import persistent_tile_scheduling_macro_amd as pg

LAYOUT = {"kn": pg.PGEMM_B_KN, "nk": pg.PGEMM_B_NK}
FEW = (cases.FEW8, cases.FEW16, cases.FEW32)
TILES = (cases.TILE64, cases.TILE128, cases.PAIR, cases.PING)


@pytest.mark.parametrize("M,N,K,layout,gated,plan", cases.PRODUCTS)
def test_products_take_the_bodies_they_name(M, N, K, layout, gated, plan):
    assert pg.pgemm_dense_query(M, N, K, LAYOUT[layout], int(gated)) == plan


@pytest.mark.parametrize("M,N,K,plan", cases.GRADIENTS)
def test_gradients_take_the_bodies_they_name(M, N, K, plan):
    assert pg.pgemm_dense_weight_grad_query(M, N, K) == plan


def test_every_body_is_reached():
    got = {(body, pieces > 1, layout, gated) for _, _, _, layout, gated, (body, pieces) in cases.PRODUCTS}
    odd = {(body, layout, gated) for _, N, K, layout, gated, (body, _) in cases.PRODUCTS if N % 8 or K % 8}
    for layout in ("kn", "nk"):
        for gated in (False, True):
            for body in FEW:
                assert (body, False, layout, gated) in got
            for body in TILES:
                assert (body, False, layout, gated) in got and (body, True, layout, gated) in got
            for body in FEW + TILES:
                assert (body, layout, gated) in odd
    grads = {(body, pieces > 1) for _, _, _, (body, pieces) in cases.GRADIENTS}
    assert grads == {(body, cut) for body in (cases.TILE128, cases.PAIR, cases.PING) for cut in (False, True)}
    for body in (cases.TILE128, cases.PAIR):
        assert any(K % 8 for _, _, K, (b, _) in cases.GRADIENTS if b == body)


def test_odd_columns_leave_the_ping_pong_body():
    """Its epilogue stores eight columns at a time."""
    for N in range(4097, 4104):
        assert pg.pgemm_dense_query(8192, N, 4096, LAYOUT["nk"])[0] != cases.PING
        assert pg.pgemm_dense_weight_grad_query(8192, 4096, N)[0] != cases.PING
    assert pg.pgemm_dense_query(8192, 4096, 4096, LAYOUT["nk"])[0] == cases.PING


def test_few_columns_of_k_by_n_weights_leave_the_few_row_body():
    """It reads four at a time."""
    for N in (1, 2, 3):
        assert pg.pgemm_dense_query(4, N, 64, LAYOUT["kn"])[0] not in FEW
        assert pg.pgemm_dense_query(4, N, 64, LAYOUT["nk"])[0] in FEW


@pytest.mark.parametrize("M,N,K,layout,plan", cases.BOTH)
def test_both_gradients_take_the_launch_they_name(M, N, K, layout, plan):
    assert pg.pgemm_dense_gradients_query(M, N, K, LAYOUT[layout]) == plan


def test_every_launch_of_both_gradients_is_reached():
    got = {(layout, body, dx > 1, dw > 1) for _, _, _, layout, (body, dx, dw) in cases.BOTH}
    assert {(layout, body) for layout, body, _, _ in got} == {(l, b) for l in LAYOUT for b in (cases.TILE128, cases.PAIR, cases.TWO)}
    assert {(dx, dw) for _, body, dx, dw in got if body != cases.TWO} == {(a, b) for a in (False, True) for b in (False, True)}
    assert any(N % 8 for _, N, _, _, (b, *_) in cases.BOTH if b != cases.TWO) and any(K % 8 for _, _, K, _, (b, *_) in cases.BOTH if b != cases.TWO)
