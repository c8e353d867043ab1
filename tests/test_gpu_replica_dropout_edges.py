"""The replica's dropout with several chunks a thread: every type, with and
without residual, rows without gaps, with gaps of one stride and of others, in
place, counters that pass a multiple of 2^32 on the way. The mask of a few rows
is the oracle's, the rest agrees with a call on fewer rows at a time."""
import numpy as np
import pytest

from oracle import replica as o
from test_gpu_replica_dropout import SEED, _seed
from test_gpu_replica_ops import FLOATS, torch, v  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS, COLS, P = 4100, 776, 0.3  # 397700 chunks, more than eight a thread of a block an SM


def _matrix(torch, pad, dtype, seed=None):  # noqa: F811
    m = torch.full((ROWS, COLS + pad), 77.0, device="cuda", dtype=getattr(torch, dtype))
    if seed is not None:
        m[:, :COLS] = torch.randn(ROWS, COLS, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    return m


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("first", [0, (1 << 32) // 97 - 2000, (5 << 32) // 97 - 7])
@pytest.mark.parametrize("xpad,rpad,ypad", [(0, 0, 0), (8, 8, 8), (0, 8, 16)])
def test_several_chunks_a_thread(torch, v, xpad, rpad, ypad, first, dtype):  # noqa: F811
    x, r, seed = _matrix(torch, xpad, dtype, 1), _matrix(torch, rpad, dtype, 2), _seed(torch)
    X, R, scale = x[:, :COLS], r[:, :COLS], 65536 / (65536 - round(P * 65536))
    for residual in (True, False):
        y, part = _matrix(torch, ypad, dtype), torch.empty(100, COLS, device="cuda", dtype=x.dtype)
        v.vrcclDropoutForward(X, R if residual else None, y[:, :COLS], ROWS, COLS, dtype, P, seed, 4, first)
        assert (y[:, COLS:] == 77).all()
        for at in range(0, ROWS, 100):  # (fewer chunks: one a thread)
            v.vrcclDropoutForward(X[at:at + 100], R[at:at + 100] if residual else None, part, 100, COLS, dtype, P, seed, 4, first + at)
            assert torch.equal(part, y[at:at + 100, :COLS]), at
        for at in (0, 1997, ROWS - 5):
            kept, _ = o.dropout_mask(5, COLS, P, SEED, 4, first + at)
            want = np.where(kept, X[at:at + 5].double().cpu().numpy() * scale, 0) + (R[at:at + 5].double().cpu().numpy() if residual else 0)
            # the scale is rounded, the sum, and the result to its type
            size = np.abs(X[at:at + 5].double().cpu().numpy()) * scale + (np.abs(R[at:at + 5].double().cpu().numpy()) if residual else 0)
            tol = 1.01 * torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2 * 2.0 ** -24 * size + 2.0 ** -24 * (dtype == "float16")
            assert (np.abs(y[at:at + 5, :COLS].double().cpu().numpy() - want) <= tol).all()
    over = r.clone()
    v.vrcclDropoutForward(X, R, y[:, :COLS], ROWS, COLS, dtype, P, seed, 4, first)
    v.vrcclDropoutForward(X, over[:, :COLS], over[:, :COLS], ROWS, COLS, dtype, P, seed, 4, first)
    assert torch.equal(over[:, :COLS], y[:, :COLS]) and (over[:, COLS:] == 77).all()
    v.vrcclDropoutBackward(X, y[:, :COLS], ROWS, COLS, dtype, P, seed, 4, first)
    v.vrcclDropoutBackward(X, X, ROWS, COLS, dtype, P, seed, 4, first)
    assert torch.equal(X, y[:, :COLS]) and (x[:, COLS:] == 77).all()
