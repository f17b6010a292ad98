"""Routing by scores and its gradient against the 64-bit forms."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import abi, say

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
LOWEST = float(np.finfo(np.float32).min)


def cuda(a, dtype=torch.float32):
    return None if a is None else torch.tensor(np.asarray(a)).to(dtype).cuda()


def make(T, E, bias, seed, ties=False):
    rng = np.random.default_rng(seed)
    logits = (rng.normal(size=(T, E)) + 0.5 * rng.normal(size=E)).astype(np.float32)
    if ties:
        logits = np.round(logits * 4) / 4
    return logits, (0.1 * rng.normal(size=E)).astype(np.float32) if bias else None


def check(logits, K, bias=None, **kw):
    ids, w = abi.route_scored(cuda(logits), K, bias=cuda(bias), **kw)
    again, w2 = abi.route_scored(cuda(logits), K, bias=cuda(bias), **kw)
    want, ww, gap = ref.route(logits.astype(np.float64), K,
                              None if bias is None else bias.astype(np.float64), **kw)
    assert gap > 1e-13  # 64-bit arithmetic on either side makes the same choices
    assert np.array_equal(ids.cpu().numpy(), want)
    got = ref.f64(w)
    tol = ref.route_tolerance(logits, want, ww, kw.get("score", "softmax"))
    assert (np.abs(got - ww) <= tol).all(), np.max(np.abs(got - ww) / (tol + 1e-300))
    assert torch.equal(ids, again) and torch.equal(w, w2)
    return want, ww


#         T    E    K  groups keep top
SHAPES = [(1, 1, 1, 1, 1, 1), (3, 7, 7, 1, 1, 1), (4, 128, 8, 1, 1, 1), (70, 256, 8, 8, 4, 2),
          (70, 256, 6, 8, 3, 1), (65, 129, 6, 3, 2, 2), (33, 512, 10, 1, 1, 1),
          (33, 512, 10, 8, 4, 2), (9, 1024, 64, 64, 33, 2), (9, 1000, 10, 4, 1, 1),
          (17, 65, 4, 5, 2, 2), (40, 16, 3, 16, 5, 1), (130, 60, 4, 4, 4, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_choices_and_weights(shape, bias, score):
    T, E, K, groups, keep, top = shape
    say(f"[scored] {shape} bias={bias} {score}")
    logits, b = make(T, E, bias, seed=E + T)
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        check(logits, K, b, score=score, groups=groups, keep=keep, group_top=top, renorm=renorm,
              scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("E", [64, 256])
def test_equal_scores_go_to_the_lower_index(score, groups, keep, top, E):
    say(f"[scored] ties {score} {groups} {keep} {top} {E}")
    logits, _ = make(50, E, False, seed=1, ties=True)
    logits[0] = 0.25
    logits[1, ::2] = logits[1, 1::2]
    check(logits, 8, None, score=score, groups=groups, keep=keep, group_top=top)
    bias = np.repeat(np.float32([0.25, 0.5]), E // 2)
    check(logits, 8, bias, score=score, groups=groups, keep=keep, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_choices_below_the_resolution_of_fp32(score, groups):
    """score + bias of neighbours apart by 1e-10 to 1e-8, in both directions"""
    say(f"[scored] near ties {score} {groups}")
    rng = np.random.default_rng(6)
    T, E = 60, 64
    logits = (rng.normal(size=(T, E)) * 0.5).astype(np.float32)
    # one bias vector that puts c of every expert of row 0 near 1/2, to fp32's steps
    s = np.exp(ref.log_scores(logits[:1].astype(np.float64), score))[0]
    bias = (0.5 - s).astype(np.float32)
    logits[1:] = logits[0]
    # rows differ from row 0 in single logits, by steps
    for t in range(1, T):
        e = t % E
        logits[t, e] = np.nextafter(logits[t, e], np.float32(9 if t % 2 else -9))
    want, _ = check(logits, 8, bias, score=score, groups=groups, keep=max(1, groups // 2),
                    group_top=2)
    c = s + bias.astype(np.float64)
    assert 0 < np.ptp(c) < 2.0 ** -23


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
def test_masks(score, renorm, groups, keep):
    say(f"[scored] masks {score} {renorm} {groups}")
    E = 64
    logits, bias = make(14, E, True, seed=8)
    logits[0] = -INF                    # nothing there
    logits[1] = NAN
    logits[2, 3:] = -INF                # fewer than K
    logits[3, ::2] = NAN
    logits[4] = LOWEST                  # the lowest value is a logit like any other
    logits[5, :50] = LOWEST
    logits[6, 5] = 3e38
    logits[7] = -120.0                  # sigmoids that fp32 does not hold
    logits[7, 9] = -119.0
    logits[8] = 90.0 + np.arange(E) / 4
    logits[9] = -1000.0 + np.arange(E)
    logits[10, 16:] = -INF              # whole groups gone
    logits[11, 7], logits[11, 9] = INF, -INF
    logits[12, 40], logits[12, 11] = INF, INF
    logits[13, :63] = -INF              # one expert
    kw = dict(score=score, renorm=renorm, groups=groups, keep=keep, group_top=2, scale=1.5)
    # (rows whose sigmoids are one or next to it differ by less than 64-bit steps
    # without a bias: left to the next test)
    rows = [t for t in range(14) if not (score == "sigmoid" and t == 8)]
    check(logits[rows], 6, None, **kw)
    bias[3], bias[20], bias[33] = -INF, NAN, 0.0
    rows = [t for t in rows if t not in (4, 5, 7, 9)]
    check(logits[rows], 6, bias, **kw)


def test_sigmoids_next_to_one_keep_their_order():
    """without a bias and groups the order is the logits' own"""
    say("[scored] saturated")
    logits = (30.0 + np.arange(128) / 2)[None].astype(np.float32).repeat(3, axis=0)
    logits[1] = logits[1, ::-1]
    ids, w = abi.route_scored(cuda(logits), 5, score="sigmoid")
    assert ids[0].tolist() == [127, 126, 125, 124, 123] and ids[1].tolist() == [0, 1, 2, 3, 4]
    assert torch.allclose(w, torch.full_like(w, 0.2))


def test_a_bias_of_infinity_is_picked_first():
    say("[scored] bias inf")
    logits, bias = make(5, 32, True, seed=2)
    bias[[7, 21]] = INF
    want, _ = check(logits, 4, bias, score="sigmoid")
    assert (want[:, 0] == 7).all() and (want[:, 1] == 21).all()


@pytest.mark.parametrize("E", [16, 64, 130, 256, 512, 1024])
def test_many_rows(E):
    say(f"[scored] many rows {E}")
    T, K = 20011, 4
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn((T, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
    c = torch.sigmoid(logits.double()) + bias.double()
    want = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :K]
    ids, w = abi.route_scored(logits, K, bias=bias, score="sigmoid", renorm=False)
    assert torch.equal(ids.long(), want)
    s = torch.gather(torch.sigmoid(logits.double()), 1, want)
    assert ((w.double() - s).abs() <= s * 60 * ref.U32).all()


# ---------------------------------------------------------------- gradient --

def check_backward(logits, ids, dw, dtype=torch.float32, add=None, inplace=False, **kw):
    a = None if add is None else cuda(add, dtype)
    wide = None if a is None else ref.f64(a)
    args = (cuda(logits), cuda(ids, torch.int32), cuda(dw))
    if inplace:
        got = abi.route_scored_backward(*args, add=a, out=a, **kw)
        assert got is a
    else:
        got = abi.route_scored_backward(*args, add=a, out_dtype=dtype, **kw)
        assert torch.equal(got, abi.route_scored_backward(*args, add=a, out_dtype=dtype, **kw))
    want, mag = ref.route_backward(logits.astype(np.float64), ids, dw.astype(np.float64), add=wide, **kw)
    tol = ref.backward_tolerance(logits, mag, want, dtype)
    off = np.abs(ref.f64(got) - want)
    assert (off <= tol).all(), np.max(off / (tol + 1e-300))


MODES = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 7, 7), (129, 64, 4), (65, 129, 6), (40, 512, 10),
                                   (7, 1024, 64), (30, 260, 3)])
def test_gradient(T, E, K, dtype, score, renorm):
    say(f"[scored] gradient {T} {E} {K} {dtype} {score} {renorm}")
    rng = np.random.default_rng(E)
    logits, _ = make(T, E, False, seed=E + 1)
    ids = np.argsort(-logits, axis=1)[:, :K].astype(np.int32)
    dw = rng.normal(size=(T, K)).astype(np.float32)
    kw = dict(score=score, renorm=renorm, scale=2.5)
    check_backward(logits, ids, dw, dtype, **kw)
    check_backward(logits, ids, dw, dtype, add=rng.normal(size=(T, E)), **kw)
    check_backward(logits, ids, dw, dtype, add=rng.normal(size=(T, E)), inplace=True, **kw)


@pytest.mark.parametrize("score,renorm", MODES)
def test_gradient_of_odd_rows(score, renorm):
    say(f"[scored] odd gradient {score} {renorm}")
    rng = np.random.default_rng(9)
    T, E, K = 12, 40, 5
    logits, _ = make(T, E, False, seed=5)
    ids = np.argsort(-logits, axis=1)[:, :K].astype(np.int32)
    dw = rng.normal(size=(T, K)).astype(np.float32)
    ids[0] = -1                          # no entry
    ids[1] = [3, -1, 3, 7, 3]            # one expert three times
    ids[2, 1:] = [E, -7, 2 ** 31 - 1, -(2 ** 31)]
    logits[3], ids[3] = -INF, [0, 1, 2, 3, 4]
    logits[4, 5:], ids[4] = NAN, [0, 1, 2, 30, 31]   # two of the entries are absent
    logits[5], logits[5, 4] = LOWEST, 0.0
    ids[5] = [4, 0, 1, 2, 3]
    logits[6] = -300.0
    ids[6] = [0, 1, 2, 3, 4]
    logits[7, 8], ids[7, 0] = INF, 8
    logits[8, 8], logits[8, 9] = INF, INF
    ids[8] = [8, 9, 1, 2, 3]
    logits[9, :3], ids[9] = 200.0, [0, 1, 5, 6, 7]
    dw[0], dw[2, 1:] = NAN, INF          # of entries that lead nowhere
    check_backward(logits, ids, dw, score=score, renorm=renorm, scale=0.5)


@pytest.mark.parametrize("E", [512, 513])
def test_offsets_past_32_bits(E):
    """2^31 logits and more: the last tokens' rows as in a call of their own"""
    say(f"[route_scored] many tokens {E}")
    T, K, n = (1 << 31) // 512 + 5, 2, 300
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.zeros((T, E), device="cuda")
    logits[:, 3], logits[:, 70] = 2.0, 1.0
    logits[-n:] = torch.randn((n, E), generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    dw = torch.rand((T, K), generator=g, device="cuda")
    kw = dict(bias=bias, score="sigmoid")
    ids, w = abi.route_scored(logits, K, **kw)
    last = logits[-n:].clone()
    few_ids, few_w = abi.route_scored(last, K, **kw)
    assert torch.equal(ids[-n:], few_ids) and torch.equal(w[-n:], few_w)
    got = abi.route_scored_backward(logits, ids, dw, renorm=False, out_dtype=torch.bfloat16)
    assert torch.equal(got[-n:], abi.route_scored_backward(
        last, few_ids, dw[-n:].clone(), renorm=False, out_dtype=torch.bfloat16))
    del got
    add = torch.ones((T, E), device="cuda")  # onto another gradient, in place
    assert abi.route_scored_backward(logits, ids, dw, renorm=False, add=add, out=add) is add
    assert torch.equal(add[-n:], abi.route_scored_backward(
        last, few_ids, dw[-n:].clone(), renorm=False, add=torch.ones((n, E), device="cuda")))
