"""moe_balance_loss and moe_route_backward on the GPU against the 64-bit forms:
counts exactly, losses and gradients within rounding bounds; padded tokens,
rows without a logit, bad and repeated ids, every width variant."""
import numpy as np
import pytest
import torch

import dense_ref as ref
from gpu_util import abi, say, synth

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(T, E, K, seed=0, empty=0.0, spread=1.0):
    g = np.random.default_rng(seed + 7 * T + E)
    logits = (g.standard_normal((T, E)) * spread).astype(np.float32)
    ids, w = abi.route(torch.from_numpy(logits).cuda(), K)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    if empty:
        ids[g.random(T) < empty] = -1
    return g, logits, ids, w


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(T, E, K, logits, ids, w, g, out="f32"):
    say(f"[balance] T={T} E={E} K={K} {out}")
    L64 = logits.astype(np.float64)
    want, cnt, prob = ref.balance(L64, ids)
    ws = torch.full((abi.moe_balance_workspace(T, E, K),), 0xFF, dtype=torch.uint8, device="cuda")
    got, _ = abi.balance_loss(dev(logits), dev(ids), workspace=ws)
    torch.cuda.synchronize()
    assert np.array_equal(got["cnt"].cpu().numpy(), cnt)
    # a probability: exp of a difference of logits (rounded: range * 2^-24), a
    # sum of E terms and a product; then additions over a group's rows, a
    # workgroup's groups and the workgroups
    fin = np.where(np.isfinite(L64), L64, 0.0)
    span = float(fin.max() - fin.min()) + 1
    adds = T // 512 + 32 + 64 + 16
    rel = (span + E + adds + 16) * ref.U32
    assert np.all(np.abs(ref.f64(got["prob"]) - prob) <= rel * prob + 1e-30)
    loss = ref.f64(got["loss"])
    # the z loss: lse is off by 2^-24 of its size and its parts', squared
    big = float(np.abs(fin).max()) + np.log(E) + 1
    assert abs(loss[0] - want[0]) <= (rel + 8 * ref.U32) * want[0] + 1e-30, (loss, want)
    ztol = 2 * big * (big + E + 8) * ref.U32 + (adds + 8) * ref.U32 * want[1]
    assert abs(loss[1] - want[1]) <= ztol, (loss, want)

    dw = g.standard_normal((T, K)).astype(np.float32)
    dl = np.array([0.3 * T, 0.02 * T], np.float32)
    for a, b in ((dw, dl), (None, dl), (dw, None)):
        d64, l64 = (None if v is None else v.astype(np.float64) for v in (a, b))
        ref_d, size = ref.route_backward(L64, ids, w.astype(np.float64), d64, cnt, l64)
        got_d = abi.route_backward(dev(logits), dev(ids), dev(w), None if a is None else dev(a),
                                   got["cnt"], None if b is None else dev(b), out_dtype=DT[out])
        torch.cuda.synchronize()
        tol = (span + E + K + 32) * ref.U32 * size
        tol = tol + ref.HALF[DT[out]] * (np.abs(ref_d) + tol) + ref.TINY[DT[out]]
        err = np.abs(ref.f64(got_d) - ref_d)
        assert np.all(err <= tol), float((err - tol).max())


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (2, 9, 9), (64, 8, 2), (3, 16, 4),
                                   (65, 17, 3), (100, 32, 5), (33, 33, 33), (257, 64, 64),
                                   (50, 65, 8), (130, 128, 6), (99, 129, 6), (300, 256, 8),
                                   (41, 257, 10), (2048, 512, 10), (20, 513, 4), (77, 1000, 12),
                                   (65, 1024, 64), (5000, 60, 4)])
def test_balance_and_gradient(T, E, K):
    g, logits, ids, w = make(T, E, K)
    check(T, E, K, logits, ids, w, g, out=("f32", "f16", "bf16")[(T + E) % 3])


@pytest.mark.parametrize("empty", [0.2, 1.0])
def test_padded_tokens(empty):
    g, logits, ids, w = make(400, 48, 4, empty=empty)
    check(400, 48, 4, logits, ids, w, g)
    if empty == 1.0:
        got, _ = abi.balance_loss(dev(logits), dev(ids))
        assert not got["loss"].any() and not got["prob"].any() and not got["cnt"].any()


def test_skipped_bad_and_repeated_ids():
    """tail-skipped slots, ids outside [0, E) and an id twice in a row of picks"""
    g, logits, ids, w = make(150, 40, 6)
    ids[g.random(ids.shape) < 0.3] = -1
    ids[::7, 2] = 40
    ids[::5, 3] = -77
    ids[::4, 1] = ids[::4, 0]
    w[::9] = 0.0
    w[ids < 0] = np.nan  # not used there
    check(150, 40, 6, logits, ids, np.where(ids < 0, 0, w), g)
    got = abi.route_backward(dev(logits), dev(ids), dev(w), dev(np.ones_like(w)),
                             dev(ref.counts(ids, 40).astype(np.int32)), None)
    assert torch.isfinite(got).all()


def test_masked_logits():
    """-inf and NaN logits are absent experts, a row of only such is empty; the
    type's lowest value is an ordinary logit"""
    g, logits, ids, w = make(64, 24, 3)
    logits[:, 5] = -np.inf
    logits[3, 7] = np.nan
    logits[8, 1:] = -np.inf
    logits[9, :] = np.finfo(np.float32).min
    logits[10, :12] = np.finfo(np.float32).min
    ids2, w2 = abi.route(dev(logits), 3)
    check(64, 24, 3, np.where(logits < -1e30, np.where(np.isinf(logits), -np.inf, -1e4), logits).astype(np.float32),
          ids2.cpu().numpy(), w2.cpu().numpy(), g)
    logits[11] = -np.inf
    logits[12] = np.nan
    ids[11], ids[12] = (0, 1, 2), (3, 4, 5)  # made-up picks of rows that have no logit
    got, _ = abi.balance_loss(dev(logits), dev(ids))
    d = abi.route_backward(dev(logits), dev(ids), dev(w), None, got["cnt"],
                           dev(np.array([1, 1], np.float32)))
    torch.cuda.synchronize()
    assert torch.isfinite(got["prob"]).all() and torch.isfinite(got["loss"][0])
    gone = np.arange(64) != 9  # (row 9 has a logit there, the lowest value)
    assert not d[11].any() and not d[12].any() and not d[gone, 5].any()
    want = ref.balance(np.where(np.isnan(logits), -np.inf, logits.astype(np.float64)), ids)
    # the lowest value's lse^2 is infinite in fp32: the z loss says so
    assert np.allclose(ref.f64(got["prob"]), want[2], rtol=1e-5, atol=0)
    assert torch.isinf(got["loss"][1])


def test_loss_difference_quotient():
    """the gradient against central differences of the loss that the GPU computes,
    along a random direction: third derivatives (below 3 gb + 2 gz span) times
    h^2 / 6, and the losses' own rounding over h"""
    g, logits, ids, w = make(96, 32, 4)
    v = g.standard_normal(logits.shape).astype(np.float32)
    v /= np.linalg.norm(v)
    dl = np.array([1.0, 0.1], np.float32)
    got, ws = abi.balance_loss(dev(logits), dev(ids))
    d = abi.route_backward(dev(logits), dev(ids), dev(w), None, got["cnt"], dev(dl))
    h = 0.05
    f = [float(ref.f64(abi.balance_loss(dev(logits + s * v), dev(ids))[0]["loss"]) @ dl)
         for s in (h, -h)]
    num, have = (f[0] - f[1]) / (2 * h), float((ref.f64(d) * v).sum())
    assert abs(num - have) <= h * h + 64 * ref.U32 * (abs(f[0]) + 1) / h, (num, have)


def test_same_bits_twice_and_in_a_graph():
    g, logits, ids, w = make(3000, 512, 10)
    a, b = dev(logits), dev(ids)
    dw, dl = dev(g.standard_normal(w.shape).astype(np.float32)), dev(np.array([1, 2], np.float32))
    one, ws = abi.balance_loss(a, b)
    d1 = abi.route_backward(a, b, dev(w), dw, one["cnt"], dl, out_dtype=torch.bfloat16)
    keep = {k: torch.empty_like(v) for k, v in one.items()}
    d2, wd = torch.empty_like(d1), dev(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.balance_loss(a, b, workspace=ws, **keep)
        abi.route_backward(a, b, wd, dw, keep["cnt"], dl, out=d2)
    for rep in range(3):
        for t in (*keep.values(), d2):
            t.zero_()
        ws.fill_(0x77)
        two, _ = abi.balance_loss(a, b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in one:
            assert torch.equal(one[k], keep[k]) and torch.equal(one[k], two[k]), (rep, k)
        assert torch.equal(d1, d2)


def test_configs_counts_are_the_plans():
    """cnt is moe_plan's cnt on the workloads' own routing, tail skipping included"""
    for name in ("tiny_fp32", "decode_bf16", "ubatch_bf16", "prefill_tailskip_fp16"):
        cfg = synth.CONFIGS[name]
        ids, w = synth.routing(cfg)
        logits = synth.router_logits(cfg)
        got, _ = abi.balance_loss(dev(logits), dev(ids))
        p = abi.plan(dev(ids), dev(w), cfg.E)
        torch.cuda.synchronize()
        assert torch.equal(got["cnt"][:cfg.E], p["cnt"]), name


def test_helper_refuses():
    l, i = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    for call in (lambda: abi.balance_loss(l.half(), i), lambda: abi.balance_loss(l, i.long()),
                 lambda: abi.balance_loss(l.t(), i),
                 lambda: abi.balance_loss(l, i, cnt=torch.zeros(8, dtype=torch.int32, device="cuda")),
                 lambda: abi.route_backward(l, i, l[:, :2].contiguous(), None,
                                            torch.zeros(10, dtype=torch.int32, device="cuda"), None)):
        with pytest.raises((TypeError, ValueError, abi.MoeError)):
            call()
