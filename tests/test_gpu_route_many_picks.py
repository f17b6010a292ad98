"""Routing by scores where a row's candidates are about as many as its lanes, or more: picks
close to the number of lanes, few open columns, equal logits; rows of either kind in one
wavefront. Choices and weights of every row against 64-bit arithmetic."""
import pytest
import torch

import block_ref as ref
from gpu_util import abi, say

pytestmark = pytest.mark.gpu


def choose(logits, K, bias, score, groups, keep, top):
    """(ids, scores of every expert) in 64 bits, ties to the lower index"""
    l = logits.double()
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, dim=1)
    c = s if bias is None else s + bias.double()
    T, E = l.shape
    key = l if bias is None else c
    if groups > 1:
        best = torch.sort(c.view(T, groups, -1), dim=2, descending=True)[0][..., :top].sum(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :keep]
        kept = torch.zeros((T, groups), dtype=torch.bool, device=l.device).scatter_(1, order, True)
        key = key.masked_fill(~kept.repeat_interleave(E // groups, dim=1), -float("inf"))
    return torch.sort(key, dim=1, descending=True, stable=True)[1][:, :K], s


def check(logits, K, bias=None, score="softmax", groups=1, keep=1, top=1):
    want, s = choose(logits, K, bias, score, groups, keep, top)
    for renorm in (True, False):
        ids, w = abi.route_scored(logits, K, bias=bias, score=score, groups=groups, keep=keep,
                                  group_top=top, renorm=renorm, scale=2.0)
        assert torch.equal(ids.long(), want)
        v = torch.gather(s, 1, want)
        v = 2.0 * (v / v.sum(dim=1, keepdim=True) if renorm else v)
        # arguments of the exponentials are at most 16 in size and each off by half a step,
        # the sums have at most 1,024 terms, 6 additions deep in a lane and 10 between lanes
        # at the most; a division or two
        assert float(logits.abs().max()) <= 8
        assert ((w.double() - v).abs() <= v * (2 * 16 + 24 + 8) * ref.U32).all()


def normal(T, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, E), generator=g, device="cuda").clamp(-8, 8), g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(32, 8), (64, 16), (65, 16), (128, 10), (128, 12), (256, 12),
                                 (256, 16), (250, 16), (512, 20), (512, 32), (509, 32), (1024, 40),
                                 (1024, 64), (17, 16)])
def test_picks_close_to_the_lanes(E, K, score):
    say(f"[picks] {E} {K} {score}")
    logits, g = normal(3001, E, E + K)
    check(logits, K, score=score)
    bias = 0.05 * torch.randn(E, generator=g, device="cuda")
    check(logits, K, bias, score=score)


@pytest.mark.parametrize("E,K,groups,keep,top", [(256, 10, 8, 1, 1), (256, 10, 8, 1, 2),
                                                 (128, 6, 16, 2, 2), (512, 16, 8, 1, 2),
                                                 (64, 8, 8, 1, 1), (1024, 24, 32, 2, 2)])
def test_few_open_columns(E, K, groups, keep, top):
    say(f"[picks] groups {E} {K} {groups} {keep}")
    logits, g = normal(1500, E, E + K)
    bias = 0.05 * torch.randn(E, generator=g, device="cuda")
    for b in (None, bias):
        for score in ("softmax", "sigmoid"):
            check(logits, K, b, score, groups, keep, top)


@pytest.mark.parametrize("E,K", [(64, 4), (128, 8), (256, 8), (512, 10), (1024, 8)])
def test_equal_rows_beside_others(E, K):
    """padding of zeros, rows of coarse steps and ordinary ones, in every place of a wavefront"""
    say(f"[picks] equal {E} {K}")
    logits, _ = normal(2003, E, E)
    logits[::3] = 0.0
    logits[1::7] = (logits[1::7] * 2).round() / 2
    logits[2::11, 1:] = logits[2::11, :1]
    check(logits, K)
    check(logits, K, score="sigmoid")
