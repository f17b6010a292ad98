"""The router kernels over more rows than their grids hold at once: every
workgroup takes several rounds of rows, the last one ragged. At most 256
workgroups of 1,024 threads take the losses' rows, 2,048 of 256 the gradient's."""
import numpy as np
import pytest

from test_gpu_balance import check, make

pytestmark = pytest.mark.gpu


def lanes(E):
    """lanes of a row; 4 columns a lane where rows are whole 16-byte chunks"""
    if E % 4 == 0:
        return 8 if E <= 32 else 16 if E <= 64 else 32 if E <= 128 else 64
    return 8 if E <= 8 else 16 if E <= 64 else 32 if E <= 128 else 64


@pytest.mark.parametrize("T,E,K,losses,gradient", [
    (9001, 512, 10, 3, 2), (8301, 129, 6, 3, 2), (8195, 255, 5, 3, 2), (16500, 513, 4, 5, 3),
    (33001, 60, 4, 3, 2), (33333, 33, 3, 3, 2), (17011, 100, 8, 3, 2), (66003, 8, 2, 3, 2),
    (66001, 5, 2, 3, 2), (33100, 17, 3, 3, 2)])
@pytest.mark.parametrize("empty", [0.0, 0.3])
def test_several_rounds(T, E, K, losses, gradient, empty):
    per = 256 // lanes(E)
    assert -(-T // (256 * 4 * per)) == losses and -(-T // (2048 * per)) == gradient
    g, logits, ids, w = make(T, E, K, empty=empty)
    ids[g.random(ids.shape) < 0.05] = -1  # skipped slots
    check(T, E, K, logits, ids, w, g, out=("f32", "f16", "bf16")[(T + K) % 3])


def test_every_row_counts_once():
    """equal rows: the same gradient row, bit for bit, whichever round and group took it,
    and whole sums that a row taken twice or not at all would change"""
    T, E, K = 9001, 512, 4
    g, logits, ids, w = make(T, E, K)
    row, pick, weight = logits[5].copy(), ids[5].copy(), w[5].copy()
    logits[:], ids[:], w[:] = row, pick, weight
    import torch

    from gpu_util import abi
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    got, _ = abi.balance_loss(d(logits), d(ids))
    c = got["cnt"].cpu().numpy()
    assert c[E] == T and c[E + 1] == T * K and (c[pick] == T).all() and c[:E].sum() == T * K
    dw = np.broadcast_to(g.standard_normal(K).astype(np.float32), (T, K))
    out = abi.route_backward(d(logits), d(ids), d(w), d(dw), got["cnt"],
                             d(np.array([T, 0.1 * T], np.float32)))
    assert torch.equal(out, out[:1].expand(T, E)) and bool(out.any())
