"""CPU: the operators' test sizes reach every kernel that the choosing rules can choose."""
import pytest

import operator_cases as cases
import persistent_tile_scheduling_macro_amd as pg

LAYOUT = {"kn": pg.PGEMM_B_KN, "nk": pg.PGEMM_B_NK}


@pytest.mark.parametrize("counts,K,N,layout,y,dx,dw", cases.GROUPED)
def test_grouped_sizes_take_the_bodies_they_name(counts, K, N, layout, y, dx, dw):
    R, E, nk = sum(counts), len(counts), layout == "nk"
    assert pg.pgemm_grouped_query(R, E, K, N, LAYOUT[layout]) == y
    assert pg.pgemm_grouped_query(R, E, N, K, LAYOUT["kn" if nk else "nk"]) == dx
    assert pg.pgemm_grouped_weight_grad_query(R, E, *((N, K) if nk else (K, N))) == dw


def test_every_grouped_body_is_reached():
    rows, grads = set(), set()
    for _, K, N, layout, y, dx, (body, pieces) in cases.GROUPED:
        odd = K % 8 > 0 or N % 8 > 0
        rows |= {(y, layout, odd), (dx, "kn" if layout == "nk" else "nk", odd)}
        grads.add((body, 1 if pieces == 1 else 2 if pieces < 8 else 8, odd))  # the pieces' sums are joined in two ways
    for body in cases.BODIES:
        for layout in ("kn", "nk"):
            assert (body, layout, False) in rows
            assert (body, layout, True) in rows or body == pg.PGEMM_GROUPED_PINGPONG
    for pieces in (1, 2, 8):
        assert (pg.PGEMM_GROUPED_PINGPONG, pieces, False) in grads
    for odd in (False, True):
        assert (pg.PGEMM_GROUPED_FEW_GRAD, 1, odd) in grads
    assert (pg.PGEMM_GROUPED_ANY, 1, True) in grads and (pg.PGEMM_GROUPED_ANY, 8, True) in grads
    assert (pg.PGEMM_GROUPED_ANY, 2, False) in grads


@pytest.mark.parametrize("M,N,K,E,form", cases.W4)
def test_4_bit_sizes_take_the_forms_they_name(M, N, K, E, form):
    assert pg.pgemm_w4_query(M, N, E or 1, E > 0) == form


def test_every_4_bit_form_is_reached():
    got = {(form, E > 0) for _, _, _, E, form in cases.W4}
    assert got == {((rows, blocks), experts) for rows in (4, 16, 32) for blocks in (1, 2) for experts in (False, True)}


def test_operands_that_cannot_be_copied_directly_leave_the_ping_pong_body():
    assert pg.pgemm_grouped_query(8200, 4, 1000, 2056, LAYOUT["nk"], wide=False) == pg.PGEMM_GROUPED_ANY
    assert pg.pgemm_grouped_weight_grad_query(6000, 3, 1288, 1032, wide=False) == (pg.PGEMM_GROUPED_ANY, 2)


def test_queries_refuse():
    for call in (lambda: pg.pgemm_grouped_query(0, 1, 8, 8, 0), lambda: pg.pgemm_grouped_query(8, 1, 8, 8, 2),
                 lambda: pg.pgemm_grouped_weight_grad_query(8, 0, 8, 8), lambda: pg.pgemm_w4_query(1, 0),
                 lambda: pg.pgemm_w4_query(1, 8, 1, False, 0)):
        with pytest.raises(pg.PgemmError) as e:
            call()
        assert e.value.status == pg.PGEMM_ERR_INVALID_ARG
    for call in (lambda: pg.pgemm_grouped_query(8, 1025, 8, 8, 0), lambda: pg.pgemm_grouped_weight_grad_query(2 ** 31, 1, 8, 8),
                 lambda: pg.pgemm_w4_query(1, 8, 65535, True)):
        with pytest.raises(pg.PgemmError) as e:
            call()
        assert e.value.status == pg.PGEMM_ERR_UNSUPPORTED
