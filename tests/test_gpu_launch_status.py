"""GPU: a call reports its own launches' status, not an error that an earlier HIP call of the thread left behind."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, I32 = torch.float16, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import persistent_tile_scheduling_macro_amd as pg
    with open("/proc/self/maps") as f:
        hip = ctypes.CDLL(next(line.split()[-1] for line in f if "libamdhip64" in line))
    h = pg.pgemm_create(0)
    pg.pgemm_set_stream(h, torch.cuda.current_stream())
    yield pg, h, hip
    hip.hipGetLastError()
    pg.pgemm_destroy(h)


def one(*shape, dtype=F16):
    return torch.ones(shape, dtype=dtype, device="cuda")


def calls(pg, h):
    """Every entry point that launches: its call, its output and what that has to be."""
    x, y, ids, off = one(4, 8), one(8, 8), torch.zeros((4, 2), dtype=I32, device="cuda"), torch.tensor([0, 8], dtype=I32, device="cuda")
    pos, w32 = torch.arange(8, dtype=I32, device="cuda"), one(4, 2, dtype=torch.float32)
    order, mat, out = torch.zeros(8, dtype=I32, device="cuda"), one(1, 8, 8), torch.zeros((8, 8), dtype=F16, device="cuda")
    dw, plan = torch.zeros((4, 2), device="cuda"), torch.zeros(8, dtype=I32, device="cuda")
    q, s = torch.full((8, 32), 0x99, dtype=torch.uint8, device="cuda"), one(8, 2)
    x64, big, rows = one(8, 64), one(256, 256), torch.tensor([0, 4096], dtype=I32, device="cuda")
    long, piece = one(4096, 8), torch.zeros(pg.pgemm_grouped_weight_grad_workspace(4096, 1, 8, 8), dtype=torch.uint8, device="cuda")
    c = torch.zeros((256, 256), dtype=F16, device="cuda")
    f, t = pg.PGEMM_F16, 4
    return {
        "dispatch": (lambda: pg.pgemm_moe_dispatch(h, x, 8, ids, 0, t, 2, 1, 8, f, plan[:2], order, plan, out), out, 1),
        "dispatch_backward": (lambda: pg.pgemm_moe_dispatch_backward(h, y, 8, pos, t, 2, 8, f, out), out[:4], 2),
        "combine": (lambda: pg.pgemm_moe_combine(h, y, 8, w32, pos, t, 2, 8, f, out), out[:4], 2),
        "combine_backward": (lambda: pg.pgemm_moe_combine_backward(h, x, 8, y, 8, w32, off, pos, t, 2, 1, 8, f, out, dw), dw, 8),
        "grouped": (lambda: pg.pgemm_grouped_run(h, y, 8, mat, off, out, 8, 1, 8, 8, 0, f), out, 8),
        "grouped gradient": (lambda: pg.pgemm_grouped_weight_grad(h, y, 8, y, 8, off, out, 8, 1, 8, 8, f), out, 8),
        "grouped gradient in pieces": (lambda: pg.pgemm_grouped_weight_grad(h, long, 8, long, 8, rows, out, 4096, 1, 8, 8, f, piece,
                                                                            piece.numel()), out, 4096),
        "w4": (lambda: pg.pgemm_w4_run(h, x64, 64, q, s, None, None, out, 8, 8, 64, 1, 32, 0, f), out, 64),
        "w4 of an empty sum": (lambda: pg.pgemm_w4_run(h, None, 0, None, None, None, None, out, 8, 8, 0, 1, 32, 0, f), out, 0),
        "gemm": (lambda: pg.pgemm_run(h, big, big, c, 256, 256, 256, f, pg.PGEMM_SCHED_STATIC, 0), c, 256),
        "gemm, stream-K": (lambda: pg.pgemm_run(h, big, big, c, 256, 256, 256, f, pg.PGEMM_SCHED_STREAMK, 0), c, 256),
        "gemm of an empty sum": (lambda: pg.pgemm_run(h, None, None, c, 256, 256, 0, f, pg.PGEMM_SCHED_STATIC, 0), c, 0),
    }


def test_an_older_error_is_not_a_calls_own(env):
    pg, h, hip = env
    failed = []
    for name, (call, out, want) in calls(pg, h).items():
        print(name, flush=True)
        out.fill_(7)
        torch.cuda.synchronize()
        assert hip.hipSetDevice(1 << 20) != 0  # an error of the thread, as a stray call leaves it
        try:
            call()
        except pg.PgemmError as e:
            failed.append((name, str(e)))
            continue
        finally:
            hip.hipGetLastError()
        torch.cuda.synchronize()
        assert bool((out == want).all()), name
    assert not failed, failed


def test_the_older_error_is_left_to_its_owner(env):
    pg, h, hip = env
    call = calls(pg, h)["combine"][0]
    torch.cuda.synchronize()
    assert hip.hipSetDevice(1 << 20) != 0
    kept = hip.hipPeekAtLastError()
    call()
    assert hip.hipPeekAtLastError() == kept
    hip.hipGetLastError()
