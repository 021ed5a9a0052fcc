"""GPU: refusals of the operators' C entry points with a live handle. Each is refused before any launch."""
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


def test_routing(env):
    pg, h, b = env
    bad, no = pg.PGEMM_ERR_INVALID_ARG, pg.PGEMM_ERR_UNSUPPORTED

    def dispatch(x=b, ldx=8, ids=b, it=0, T=2, k=2, E=3, H=8, dt=F16, off=b, order=b, pos=b, xs=b, work=None, wb=0):
        pg.pgemm_moe_dispatch(h, x, ldx, ids, it, T, k, E, H, dt, off, order, pos, xs, work, wb)

    for kw in ({"T": -1}, {"k": 0}, {"H": -1}, {"E": 0}, {"dt": F8}, {"it": 2}, {"ldx": -1}, {"x": None}, {"ids": None},
               {"off": None}, {"order": None}, {"pos": None}, {"xs": None}, {"T": 40000}, {"T": 40000, "work": b, "wb": 8}):
        refused(pg, bad, lambda kw=kw: dispatch(**kw))
    for kw in ({"E": 1025}, {"T": BIG}, {"H": BIG}, {"T": 2 ** 29, "k": 3}, {"T": 2 ** 27, "k": 1}):
        refused(pg, no, lambda kw=kw: dispatch(**kw))
    for kw in ((-1, 2, 8, F16), (2, 0, 8, F16), (2, 2, -1, F16), (2, 2, 8, F8)):
        T, k, H, dt = kw
        refused(pg, bad, lambda: pg.pgemm_moe_dispatch_backward(h, b, 8, b, T, k, H, dt, b))
        refused(pg, bad, lambda: pg.pgemm_moe_combine(h, b, 8, b, b, T, k, H, dt, b))
        refused(pg, bad, lambda: pg.pgemm_moe_combine_backward(h, b, 8, b, 8, b, b, b, T, k, 3, H, dt, b, b))
    refused(pg, bad, lambda: pg.pgemm_moe_dispatch_backward(h, None, 8, b, 2, 2, 8, F16, b))
    refused(pg, bad, lambda: pg.pgemm_moe_combine(h, b, 8, None, b, 2, 2, 8, F16, b))
    refused(pg, bad, lambda: pg.pgemm_moe_combine(h, b, -8, b, b, 2, 2, 8, F16, b))
    refused(pg, bad, lambda: pg.pgemm_moe_combine_backward(h, b, 8, b, 8, b, b, b, 2, 2, 3, 8, F16, b, None))
    refused(pg, bad, lambda: pg.pgemm_moe_combine_backward(h, b, -1, b, 8, b, b, b, 2, 2, 3, 8, F16, b, b))
    refused(pg, no, lambda: pg.pgemm_moe_combine(h, b, 8, b, b, BIG, 2, 8, F16, b))


def test_grouped_products(env):
    pg, h, b = env
    bad, no = pg.PGEMM_ERR_INVALID_ARG, pg.PGEMM_ERR_UNSUPPORTED

    def rows(x=b, ldx=8, w=b, off=b, y=b, R=4, E=2, K=8, N=8, layout=0, dt=F16):
        pg.pgemm_grouped_run(h, x, ldx, w, off, y, R, E, K, N, layout, dt)

    for kw in ({"R": -1}, {"E": 0}, {"K": -1}, {"N": -1}, {"ldx": -1}, {"layout": 2}, {"dt": F8}, {"x": None}, {"w": None},
               {"off": None}, {"y": None}):
        refused(pg, bad, lambda kw=kw: rows(**kw))
    for kw in ({"R": BIG}, {"E": 1025}, {"K": BIG}, {"N": BIG}, {"R": 2 ** 30, "N": 2 ** 30}):
        refused(pg, no, lambda kw=kw: rows(**kw))

    def grad(a=b, lda=8, c=b, ldb=8, off=b, out=b, R=4, E=2, I=8, J=8, dt=BF16, work=None, wb=0):
        pg.pgemm_grouped_weight_grad(h, a, lda, c, ldb, off, out, R, E, I, J, dt, work, wb)

    long = {"R": 32768, "E": 1}
    need = pg.pgemm_grouped_weight_grad_workspace(32768, 1, 8, 8)
    for kw in ({"R": -1}, {"E": 0}, {"I": -1}, {"J": -1}, {"lda": -1}, {"ldb": -1}, {"dt": F8}, {"a": None}, {"c": None},
               {"off": None}, {"out": None}, long, dict(long, work=b, wb=need - 4), dict(long, work=b.data_ptr() + 4, wb=need)):
        refused(pg, bad, lambda kw=kw: grad(**kw))
    for kw in ({"R": BIG}, {"E": 1025}, {"I": BIG}, {"J": BIG}, {"E": 1024, "I": 2 ** 30, "J": 2 ** 30}):
        refused(pg, no, lambda kw=kw: grad(**kw))


def test_4_bit_product(env):
    pg, h, b = env
    bad, no = pg.PGEMM_ERR_INVALID_ARG, pg.PGEMM_ERR_UNSUPPORTED

    def run(x=b, ldx=64, q=b, s=b, z=None, off=None, y=b, M=1, N=8, K=64, E=1, group=32, fmt=0, dt=F16):
        pg.pgemm_w4_run(h, x, ldx, q, s, z, off, y, M, N, K, E, group, fmt, dt)

    for kw in ({"M": -1}, {"N": -1}, {"K": -1}, {"E": 0}, {"ldx": -1}, {"group": 48}, {"fmt": 2}, {"dt": F8}, {"fmt": 1, "z": b},
               {"E": 2}, {"x": None}, {"q": None}, {"s": None}, {"y": None}):
        refused(pg, bad, lambda kw=kw: run(**kw))
    for kw in ({"M": BIG}, {"N": BIG}, {"K": BIG}, {"E": 65535, "off": b}, {"N": 2 ** 29}):
        refused(pg, no, lambda kw=kw: run(**kw))


def test_empty_calls_need_no_pointers(env):
    pg, h, _ = env
    pg.pgemm_moe_combine(h, None, 8, None, None, 0, 2, 8, F16, None)
    pg.pgemm_moe_dispatch_backward(h, None, 8, None, 0, 2, 8, F16, None)
    pg.pgemm_grouped_run(h, None, 8, None, None, None, 0, 2, 8, 8, 0, F16)
    pg.pgemm_grouped_weight_grad(h, None, 8, None, 8, None, None, 0, 2, 0, 8, F16)
    pg.pgemm_w4_run(h, None, 64, None, None, None, None, None, 0, 8, 64, 1, 32, 0, F16)
