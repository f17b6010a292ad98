"""Calls whose rows make a grid of 2^32 threads and more, which one launch does not hold: HIP
starts such a grid modulo 2^32, without an error. Every row is computed."""
import pytest
import torch

from gpu_util import abi, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,K", [((1 << 28) + 21, 1, 1), ((1 << 28) + 37, 4, 2)])
def test_routing_by_scores(T, E, K):
    """16 lanes a row: 2^28 rows are 2^32 threads"""
    say(f"[threads] route_scored {T} {E} {K}")
    logits = torch.zeros((T, E), device="cuda")
    logits[:, E - 1] = 1.0
    logits[T // 2:, 0] = 2.0
    ids, w = torch.full((T, K), -7, dtype=torch.int32, device="cuda"), torch.full((T, K), -7.0,
                                                                                  device="cuda")
    abi.route_scored(logits, K, ids=ids, w=w)
    for t in (0, 1, T // 2 - 1, T // 2, T - 30, T - 1):
        one, v = abi.route_scored(logits[t:t + 1].clone(), K)
        assert torch.equal(ids[t:t + 1], one) and torch.equal(w[t:t + 1], v), t
    # the rows of each half are all alike
    for part in (slice(0, T // 2), slice(T // 2, T)):
        for x in (ids, w):
            assert bool((x[part] == x[part][0]).all())
    del ids
    got = torch.full((T, E), -7.0, device="cuda")
    ids = torch.full((T, K), E - 1, dtype=torch.int32, device="cuda")
    abi.route_scored_backward(logits, ids, w, score="sigmoid", renorm=False, out=got)
    for t in (0, T // 2 - 1, T // 2, T - 1):
        one = abi.route_scored_backward(logits[t:t + 1].clone(), ids[t:t + 1].clone(),
                                        w[t:t + 1].clone(), score="sigmoid", renorm=False)
        assert torch.equal(got[t:t + 1], one), t
    for part in (slice(0, T // 2), slice(T // 2, T)):
        assert bool((got[part] == got[part][0]).all())


def test_router():
    """a wavefront a row: 2^26 rows are 2^32 threads"""
    T, E, K = (1 << 26) + 21, 3, 2
    say(f"[threads] route_topk {T}")
    logits = torch.zeros((T, E), device="cuda")
    logits[:, 2] = 1.0
    logits[T // 2:, 0] = 2.0
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), -7.0, device="cuda")
    abi.moe_route_topk(logits, T, E, K, ids, w)
    for part in (slice(0, T // 2), slice(T // 2, T)):
        one, v = abi.route(logits[part][:1].clone(), K)
        assert bool((ids[part] == one).all()) and bool((w[part] == v).all())


@pytest.mark.parametrize("T,d", [((1 << 26) + 21, 8), ((1 << 22) + 5, 4096)])
def test_combine(T, d):
    """a workgroup of 64 to 1,024 threads a token: 2^26 tokens of 8 columns, 2^22 of 4,096"""
    say(f"[threads] combine {T} {d}")
    y = torch.arange(3 * d, device="cuda", dtype=torch.float32).reshape(3, d) + 1
    pos = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    pos[T // 2:] = 2
    pos[-1] = -1
    out = torch.full((T, d), -7.0, device="cuda")
    abi.moe_combine(y, 3, pos, T, 1, d, out)
    for part, want in ((slice(0, T // 2), y[0]), (slice(T // 2, T - 1), y[2]),
                       (slice(T - 1, T), torch.zeros_like(y[0]))):
        for cut in torch.split(out[part], 1 << 20):
            assert bool((cut == want).all())


def test_gather():
    """8 threads a row: 2^29 rows are 2^32 threads"""
    n, T, d = (1 << 29) + 77, 3, 8
    say(f"[threads] gather {n}")
    x = torch.arange(T * d, device="cuda", dtype=torch.float32).reshape(T, d).to(torch.bfloat16) + 1
    stok = torch.zeros(n, dtype=torch.int32, device="cuda")
    stok[n // 2:] = 2
    stok[-3] = -1
    stok[-2] = 1
    meta = torch.zeros(abi.META_N, dtype=torch.int32, device="cuda")
    meta[2] = n - 1  # rows of the plan (MOE_META_NR): the last one stays as it is
    xs = torch.full((n, d), -7.0, dtype=torch.bfloat16, device="cuda")
    abi.moe_gather(x, abi.MOE_BF16, T, d, stok, meta, n, xs)
    for part, want in ((slice(0, n // 2), x[0]), (slice(n // 2, n - 3), x[2]),
                       (slice(n - 3, n - 2), 0 * x[0]), (slice(n - 2, n - 1), x[1]),
                       (slice(n - 1, n), torch.full_like(x[0], -7.0))):
        for cut in torch.split(xs[part], 1 << 25):
            assert bool((cut == want).all())
