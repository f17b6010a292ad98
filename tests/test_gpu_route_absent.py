"""Routing by scores where NaN or -inf logits mark whole neighbourhoods of experts absent:
a mask of a layer's neighbouring experts, as a user sets it, against the 64-bit form."""
import numpy as np
import pytest
import torch

from gpu_util import abi, say
from test_gpu_route_scored import check, cuda, make

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def lanes(E, K):
    """lanes that hold a row, by the numbers of experts and picks"""
    return 16 if K <= 16 and E <= 256 else 32 if K <= 32 and E <= 512 else 64


def runs(E, length, rng, T):
    """[T, E]: each row has one to four aligned runs of `length` experts gone"""
    gone = np.zeros((T, E), bool)
    for t in range(T):
        for _ in range(1 + t % 4):
            at = length * rng.integers(0, max(1, E // length))
            gone[t, at:at + length] = True
    return gone


def strided(E, K, rng, T):
    """[T, E]: every expert e gone whose e (or e / 4) is one of a few numbers modulo the
    lanes of a row"""
    L, gone = lanes(E, K), np.zeros((T, E), bool)
    width = 4 if E % 4 == 0 else 1
    for t in range(T):
        some = rng.choice(L, size=1 + t % (L // 2), replace=False)
        gone[t] = np.isin(np.arange(E) // width % L, some)
    return gone


#          E    K: 16, 32 and 64 lanes a row, whole 16-byte rows and odd ones
WIDTHS = [(64, 2), (64, 8), (64, 15), (128, 8), (256, 12), (67, 6), (129, 8), (256, 24), (512, 10),
          (512, 30), (509, 10), (300, 20), (1024, 8), (1024, 50), (1021, 12), (96, 40)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,K", WIDTHS)
def test_neighbours_gone(E, K, bias, score):
    say(f"[absent] {E} {K} bias={bias} {score}")
    rng = np.random.default_rng(E + K)
    T = 24
    for n, gone in enumerate([runs(E, 4, rng, T), runs(E, 8, rng, T), runs(E, 16, rng, T),
                              strided(E, K, rng, T)]):
        for mark in (NAN, -INF):
            logits, b = make(T, E, bias, seed=n + E)
            logits[gone] = mark
            if mark != mark:  # a few of the other kind beside them
                logits[:, E // 3] = -INF
            check(logits, K, b, score=score, renorm=n % 2 == 0, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,groups,keep,top", [(64, 6, 4, 2, 2), (128, 8, 8, 4, 1), (256, 8, 8, 3, 2),
                                                 (60, 4, 5, 3, 2), (512, 10, 8, 4, 2),
                                                 (1024, 12, 16, 5, 2), (96, 3, 32, 5, 1)])
def test_neighbours_gone_in_groups(E, K, groups, keep, top, score):
    say(f"[absent] groups {E} {K} {groups} {score}")
    rng = np.random.default_rng(E + groups)
    T = 24
    for n, gone in enumerate([runs(E, 4, rng, T), runs(E, 16, rng, T), runs(E, E // groups, rng, T),
                              strided(E, max(K, groups), rng, T)]):
        for bias in (False, True):
            logits, b = make(T, E, bias, seed=n + E)
            logits[gone] = NAN
            check(logits, K, b, score=score, groups=groups, keep=keep, group_top=top,
                  renorm=n % 2 == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 128, 512])
def test_as_many_experts_as_picks(E, score):
    """K experts or fewer are there, each among absent neighbours of either kind"""
    say(f"[absent] few left {E} {score}")
    for K in (2, 8):
        for mark in (NAN, -INF):
            logits = np.full((3 * K, E), mark, np.float32)
            rng = np.random.default_rng(K)
            for t in range(3 * K):
                there = rng.choice(E // 4, size=1 + t % K, replace=False) * 4 + t % 4
                logits[t, there] = rng.normal(size=len(there))
            ids, _ = check(logits, K, None, score=score)
            assert (np.sort(ids, axis=1)[:, ::-1][:, 0] >= 0).all()


@pytest.mark.parametrize("bits", [0x7fc00000, 0xffc00000, 0x7f800001, 0xff800001, 0x7fffffff])
def test_any_nan(bits):
    """quiet and signalling NaN of either sign"""
    say(f"[absent] nan {bits:x}")
    logits, _ = make(40, 64, False, seed=3)
    gone = np.random.default_rng(1).integers(0, 16, size=40)
    cols = 4 * gone[:, None] + np.arange(4)
    raw = logits.view(np.uint32)
    np.put_along_axis(raw, cols, np.uint32(bits), axis=1)
    with np.errstate(invalid="ignore"):  # (a signalling NaN widened to 64 bits)
        want, _ = check(logits, 8, None)
    got, w = abi.route_scored(torch.tensor(raw.view(np.int32)).cuda().view(torch.float32), 8)
    assert np.array_equal(got.cpu().numpy(), want)
    # the same row with -inf in their place
    np.put_along_axis(logits, cols, np.float32(-INF), axis=1)
    ids, v = abi.route_scored(cuda(logits), 8)
    assert torch.equal(ids, got) and torch.equal(v, w)
