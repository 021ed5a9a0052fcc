"""GPU: the 4-bit product in each form its rule chooses (rows at once, column blocks), against the plain form in 64 bits."""
import pytest
import torch

import operator_refs as ref
from test_gpu_w4 import DT, KINDS, check, gen, normal, values, weights, w4  # noqa: F401 (w4 is the fixture)

pytestmark = pytest.mark.gpu


def test_a_pass_stores_its_own_rows_only(w4):  # noqa: F811
    """Four rows at once and an expert of 14, in place in one workgroup: a pass that stored rows past its four would
    change what the next one reads."""
    import persistent_tile_scheduling_macro_amd as pg
    E, M, K = 8, 14, 16
    q, s, _ = weights(K, K, 32, torch.float16, False, E)
    x = normal(M, K, dtype=torch.float16, seed=1)
    off = torch.tensor([0, 0, 0, M, M, M, M, M, M], dtype=torch.int32, device="cuda")
    want = w4.matmul(x, q, s, group=32, offsets=off)
    ref.assert_within(want, *ref.grouped(x, values(q, s, None, K, 32, "int4"), off, "nk"), 2 * K + 2)
    h = pg.pgemm_create(0)
    pg.pgemm_set_stream(h, torch.cuda.current_stream())
    pg.pgemm_w4_run(h, x, K, q, s, None, off, x, M, K, K, E, 32, pg.PGEMM_W4_INT4, pg.PGEMM_F16)
    torch.cuda.synchronize()
    pg.pgemm_destroy(h)
    assert torch.equal(x, want)
