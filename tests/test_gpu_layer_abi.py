"""GPU: refusals of the linear layer's, the router's and the routed layer's C entry points with a live handle."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F8 = 0, 1, 2
BIG = 2 ** 30 + 1


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import persistent_tile_scheduling_macro_amd as pg
    h = pg.pgemm_create(0)
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    yield pg, h, buf
    pg.pgemm_destroy(h)


def refused(pg, status, call):
    with pytest.raises(pg.PgemmError) as e:
        call()
    assert e.value.status == status, str(e.value)
    assert ": " in str(e.value)  # a reason is given


def test_linear_layer(env):
    pg, h, b = env
    bad, no = pg.PGEMM_ERR_INVALID_ARG, pg.PGEMM_ERR_UNSUPPORTED

    def run(x=b, ldx=8, w=b, ldw=8, bias=None, res=None, ldr=8, y=b, z=None, M=4, N=8, K=8, layout=1, act=0, gated=0, dt=F16,
            work=None, wb=0):
        pg.pgemm_dense_run(h, x, ldx, w, ldw, bias, res, ldr, y, z, M, N, K, layout, act, gated, dt, work, wb)

    need = pg.pgemm_dense_workspace(300, 64, 4096, 1)
    assert need > 0
    cut = {"M": 300, "N": 64, "K": 4096, "ldx": 4096, "ldw": 4096}
    for kw in ({"M": -1}, {"N": -1}, {"K": -1}, {"ldx": -1}, {"ldw": -1}, {"ldr": -1}, {"layout": 2}, {"act": 5}, {"act": -1}, {"gated": 2},
               {"dt": F8}, {"x": None}, {"w": None}, {"y": None}, cut, dict(cut, work=b, wb=need - 4),
               dict(cut, work=b.data_ptr() + 4, wb=need), dict(cut, x=b.data_ptr() + 2, work=b, wb=need)):
        refused(pg, bad, lambda kw=kw: run(**kw))
    for kw in ({"M": BIG}, {"N": BIG}, {"K": BIG}, {"K": 2 ** 22}, {"M": 2 ** 29, "N": 2 ** 20}):
        refused(pg, no, lambda kw=kw: run(**kw))

    def back(dy=b, lddy=8, x=b, ldx=8, w=b, ldw=8, z=None, dx=b, dw=b, db=b, M=4, N=8, K=8, layout=1, act=0, gated=0, dt=BF16, work=b,
             wb=1 << 20):
        pg.pgemm_dense_backward(h, dy, lddy, x, ldx, w, ldw, z, dx, dw, db, M, N, K, layout, act, gated, dt, work, wb)

    for kw in ({"M": -1}, {"N": -1}, {"K": -1}, {"lddy": -1}, {"ldx": -1}, {"ldw": -1}, {"layout": -1}, {"act": 7}, {"gated": -1},
               {"dt": F8}, {"dy": None}, {"x": None}, {"w": None}, {"act": 4}, {"gated": 1}, {"wb": 8}, {"work": None}):
        refused(pg, bad, lambda kw=kw: back(**kw))
    for kw in ({"M": BIG}, {"N": 2 ** 22}, {"K": 2 ** 22}):
        refused(pg, no, lambda kw=kw: back(**kw))


def test_router_and_layer(env):
    pg, h, b = env
    bad, no = pg.PGEMM_ERR_INVALID_ARG, pg.PGEMM_ERR_UNSUPPORTED

    def route(l=b, ld=8, ty=3, T=2, E=8, k=2, score=0, norm=1, ids=b, w=b):
        pg.pgemm_moe_route(h, l, ld, ty, T, E, k, score, norm, ids, w)

    def back(d=b, l=b, ld=8, ty=0, ids=b, w=b, T=2, E=8, k=2, score=0, norm=1, dl=b):
        pg.pgemm_moe_route_backward(h, d, l, ld, ty, ids, w, T, E, k, score, norm, dl)

    for call in (route, back):
        for kw in ({"T": -1}, {"E": 0}, {"k": 0}, {"k": 9}, {"ld": -1}, {"ty": 2}, {"score": 2}, {"norm": 2}, {"l": None}, {"ids": None},
                   {"w": None}):
            refused(pg, bad, lambda kw=kw: call(**kw))
        for kw in ({"T": 2 ** 24 + 1}, {"E": 1025}, {"E": 500, "k": 65}):
            refused(pg, no, lambda kw=kw: call(**kw))
    refused(pg, bad, lambda: back(d=None))
    refused(pg, bad, lambda: back(dl=None))

    def layer(x=b, ldx=8, ids=b, it=0, w=b, w_in=b, w_out=b, out=b, T=2, k=2, E=3, H=8, I=6, act=4, gated=1, dt=F16, work=b, wb=1 << 20):
        pg.pgemm_moe_layer(h, x, ldx, ids, it, w, w_in, w_out, out, T, k, E, H, I, act, gated, dt, work, wb)

    for kw in ({"T": -1}, {"k": 0}, {"E": 0}, {"H": -1}, {"I": -1}, {"ldx": -1}, {"it": 2}, {"act": 5}, {"gated": 2}, {"dt": F8}, {"x": None},
               {"ids": None}, {"w": None}, {"w_in": None}, {"w_out": None}, {"out": None}, {"work": None}, {"wb": 100},
               {"work": b.data_ptr() + 8}):
        refused(pg, bad, lambda kw=kw: layer(**kw))
    for kw in ({"T": 4097}, {"k": 33}, {"E": 1025}, {"H": 2 ** 21}, {"I": 2 ** 20}):
        refused(pg, no, lambda kw=kw: layer(**kw))


def test_empty_calls_need_no_pointers(env):
    pg, h, b = env
    pg.pgemm_dense_run(h, None, 8, None, 8, None, None, 0, None, None, 0, 8, 8, 1, 0, 0, F16)
    pg.pgemm_dense_run(h, None, 8, None, 8, None, None, 0, None, None, 4, 0, 8, 1, 0, 0, F16)
    pg.pgemm_dense_backward(h, None, 8, None, 8, None, 8, None, None, None, None, 4, 8, 8, 1, 0, 0, F16)
    pg.pgemm_moe_route(h, None, 8, 3, 0, 8, 2, 0, 1, None, None)
    pg.pgemm_moe_layer(h, None, 8, None, 0, None, None, None, None, 0, 2, 3, 8, 6, 0, 0, F16)
