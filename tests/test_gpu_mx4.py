"""Expert weights in microscaled 4-bit floating point: quantisation, the way back, and
the routed layer computed from them."""
import numpy as np
import pytest
import torch

import block_ref as ref
import oracle
from gpu_util import TOL, TORCH16, abi, custom, dev, host, make_case, rel_err, say, synth
from test_gpu_packed import BIG, CASES as PACKED_CASES

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
SHAPES = [(1, 8, 8), (2, 40, 72), (3, 32, 256), (2, 96, 264), (1, 328, 520), (5, 64, 64),
          (1, 200, 1032), (7, 8, 24)]


def shaped(E, d, f, kind):
    return (E, d, f) if kind == "gate" else (E, f, d)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("kind", ["gate", "down"])
@pytest.mark.parametrize("E,d,f", SHAPES)
def test_codes_scales_and_values(E, d, f, kind, dtype):
    say(f"[mx4] {E} {d} {f} {kind} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(d + f)
    w = torch.randn(shaped(E, d, f, kind), generator=g, device="cuda")
    w = (w * torch.exp(2 * torch.randn(w.shape, generator=g, device="cuda"))).to(dtype)
    w[0, 0, :4] = torch.tensor([0.0, -0.0, 6.0, -0.25])
    packed = abi.mx4_quantize(w, kind, packed=torch.full(
        (abi.moe_mx4_weight_bytes(E, d, f, abi.MX4_KINDS[kind]),), 0xA5, dtype=torch.uint8,
        device="cuda"))
    Kd, N = w.shape[1:]
    codes, scales = ref.mx4_encode(ref.f64(w))
    got, gs = ref.mx4_unpack(packed.cpu().numpy(), E, Kd, N, kind == "down")
    assert np.array_equal(gs, scales)
    assert np.array_equal(got, codes)
    # what lies past d and f is zero
    code, _, size = ref.mx4_places(Kd, N, kind == "down")
    m = 2 if kind == "down" else 1
    whole = ref.mx4_places(-(-Kd // 32) * 32, -(-N // (256 * m)) * 256 * m, kind == "down")
    assert whole[2] == size
    k = np.arange(whole[0].shape[0])[:, None]
    nib = (packed.cpu().numpy().reshape(E, size)[:, whole[0]] >> (k % 2 * 4)) & 15
    nib[:, :Kd, :N] = 0
    assert not nib.any()
    values = ref.mx4_values(codes, scales)
    for D in (F32, F16, BF16):
        back = abi.mx4_dequantize(packed, E, d, f, kind, dtype=D)
        assert torch.equal(back.cpu(), torch.tensor(values).to(D))
        assert torch.equal(torch.signbit(back.cpu()), torch.tensor((codes & 8) != 0))
    # values of the format are kept
    again = abi.mx4_quantize(abi.mx4_dequantize(packed, E, d, f, kind, dtype=F32), kind)
    assert torch.equal(abi.mx4_dequantize(again, E, d, f, kind, dtype=F32),
                       abi.mx4_dequantize(packed, E, d, f, kind, dtype=F32))


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
def test_extremes(dtype):
    say(f"[mx4] extremes {dtype}")
    big = float(torch.finfo(dtype).max)
    w = torch.randn((1, 96, 64), device="cuda").to(dtype)
    w[0, :32, 0] = 0
    w[0, 3, 1] = float("inf")
    w[0, 4, 2] = float("nan")
    w[0, :32, 3] = big
    w[0, :32, 4] = -big
    w[0, :32, 5] = float(torch.finfo(dtype).tiny)
    w[0, :32, 6] = float(torch.finfo(dtype).smallest_normal) / 4
    w[0, 32:64, 7] *= 2.0 ** -14
    w[0, 40, 8] = -float("inf")
    packed = abi.mx4_quantize(w, "gate")
    codes, scales = ref.mx4_encode(ref.f64(w))
    got, gs = ref.mx4_unpack(packed.cpu().numpy(), 1, 96, 64, False)
    assert np.array_equal(gs, scales) and (gs == 255).sum() == 3
    fine = np.repeat(scales != 255, 32, axis=1)
    assert np.array_equal(got[fine], codes[fine])
    for D in (F32, F16, BF16):
        back = abi.mx4_dequantize(packed, 1, 96, 64, "gate", dtype=D).cpu()
        want = torch.tensor(ref.mx4_values(codes, scales)).to(D)
        assert torch.equal(back.isnan(), want.isnan())
        assert torch.equal(back[~want.isnan()], want[~want.isnan()])


def test_every_scale_byte():
    """blocks whose scale is any byte, all codes, read back in each type"""
    say("[mx4] scales")
    code, scale, size = ref.mx4_places(32, 256, False)
    p = np.zeros((1, size), np.uint8)
    codes = (np.arange(32)[:, None] + np.arange(256)[None, :]) % 16
    np.bitwise_or.at(p[0], code, (codes << (np.arange(32)[:, None] % 2 * 4)).astype(np.uint8))
    p[0, scale[0]] = np.arange(256)
    packed = torch.tensor(p.reshape(-1)).cuda()
    values = ref.mx4_values(codes[None], np.arange(256, dtype=np.uint8)[None, None])
    for D in (F32, F16, BF16):
        back = abi.mx4_dequantize(packed, 1, 32, 256, "gate", dtype=D).cpu()
        want = torch.tensor(values).to(D)
        assert torch.equal(back.isnan(), want.isnan())
        assert torch.equal(back[~want.isnan()], want[~want.isnan()])


# ------------------------------------------------------------------- layer --

def four_bits(case):
    """(packed 4-bit weights, their values as the case's type)"""
    cfg = case.cfg
    ws = {"gate": ("wg", "gate"), "up": ("wu", "gate"), "down": ("wd", "down")}
    packed, values = {}, {}
    for k, (name, kind) in ws.items():
        packed[k] = abi.mx4_quantize(case.d(name), kind)
        values[k] = abi.mx4_dequantize(packed[k], cfg.E, cfg.d, cfg.f, kind,
                                       dtype=TORCH16[cfg.dtype])
    return packed, values


def four_calls(x, ids, w, values, cfg):
    """plan, gather, grouped FFN and combine one by one, with packed weights"""
    T, K = ids.shape
    D = abi.DTYPE_NAME[cfg.dtype]
    pk = abi.pack(values["gate"], values["up"], values["down"])
    p = abi.plan(ids, w, cfg.E, cfg.tm)
    n = p["sizes"].max_rows
    xs = torch.zeros((n, cfg.d), dtype=x.dtype, device="cuda")
    h = torch.zeros((n, cfg.f), dtype=x.dtype, device="cuda")
    y = torch.zeros((n, cfg.d), dtype=F32, device="cuda")
    out = torch.empty((T, cfg.d), dtype=F32, device="cuda")
    abi.moe_gather(x, D, T, cfg.d, p["stok"], p["meta"], n, xs)
    scratch = torch.empty(abi.moe_ffn_scratch_bytes(cfg.E, cfg.d, cfg.f, cfg.tm, n, D),
                          dtype=torch.uint8, device="cuda")
    abi.moe_expert_ffn_packed(xs, pk["gate"], pk["up"], pk["down"], D, cfg.E, cfg.d, cfg.f, cfg.tm,
                              p["eoff"], p["stok"], p["sw"], p["meta"], n, h, y, scratch)
    abi.moe_combine(y, n, p["pos"], T, K, cfg.d, out)
    return out


LAYERS = [c for c in PACKED_CASES if c.dtype != "f32"] + [
    custom("one_token_bf16", T=1, d=264, E=8, K=2, f=136, dtype="bf16", x_std=1.0),
    custom("one_token_f16", T=1, d=2816, E=16, K=8, f=704, dtype="f16", x_std=1.0),
]


def reference(case, ids, values):
    """(out [T, d], how far it may be off) in 64 bits. Products are summed in fp32 (at most
    d or f terms one after another), silu has 16 roundings' worth, h is rounded once to the
    type, y to fp32 and, for bf16, to binary16 with an exponent per block."""
    cfg = case.cfg
    U, half = ref.U32, ref.HALF[TORCH16[cfg.dtype]]
    x = ref.f64(case.d("x"))
    wg, wu, wd = (ref.f64(values[k]) for k in ("gate", "up", "down"))
    out, tol = np.zeros((cfg.T, cfg.d)), np.zeros((cfg.T, cfg.d))
    for e in range(cfg.E):
        t, k = np.nonzero(ids == e)
        if not len(t):
            continue
        g, u = x[t] @ wg[e], x[t] @ wu[e]
        eg, eu = ((np.abs(x[t]) @ np.abs(m[e])) * cfg.d * U for m in (wg, wu))
        sig = 1 / (1 + np.exp(-g))
        h = g * sig * u
        eh = np.abs(h) * (half + 16 * U) + (1.1 * eg * np.abs(u) + np.abs(g * sig) * eu) + 2.0 ** -25
        w = case.w[t, k][:, None].astype(np.float64)
        y = h @ wd[e]
        ey = eh @ np.abs(wd[e]) + (np.abs(h) @ np.abs(wd[e])) * cfg.f * U
        ey += (2.0 ** -11 if cfg.dtype == "bf16" else U) * (np.abs(y) + ey) + U * np.abs(y)
        np.add.at(out, t, w * y)
        np.add.at(tol, t, w * (ey + (cfg.K + 2) * U * np.abs(y)))
    return out, tol + 2.0 ** -40 * np.abs(out).max()


@pytest.mark.parametrize("cfg", LAYERS, ids=lambda c: c.name)
def test_layer(cfg):
    say(f"[mx4] layer {cfg.name}")
    case = make_case(cfg)
    packed, values = four_bits(case)
    x, ids, w = case.d("x"), case.d("ids"), case.d("w")
    out, ws = abi.forward_mx4(x, ids, w, packed, cfg.E, cfg.f, tm=cfg.tm, out_dtype=F32)
    want, tol = reference(case, case.ids, values)
    off = np.abs(ref.f64(out) - want)
    assert (off <= tol).all(), np.max(off / tol)
    # the output's type: one rounding of the same sums; another workspace's contents
    ws.fill_(0xC3)
    half, _ = abi.forward_mx4(x, ids, w, packed, cfg.E, cfg.f, tm=cfg.tm, workspace=ws)
    assert torch.equal(half, out.to(x.dtype))


@pytest.mark.parametrize("cfg", [c for c in BIG if c.dtype != "f32"], ids=lambda c: c.name)
def test_layer_of_many_rows_is_the_packed_layer_on_the_values(cfg):
    say(f"[mx4] layer bits {cfg.name}")
    case = make_case(cfg)
    packed, values = four_bits(case)
    x, ids, w = case.d("x"), case.d("ids"), case.d("w")
    out, _ = abi.forward_mx4(x, ids, w, packed, cfg.E, cfg.f, tm=cfg.tm, out_dtype=F32)
    if cfg.dtype == "bf16":
        want, _ = abi.forward(x, ids, w, values["gate"], values["up"], values["down"], tm=cfg.tm,
                              packed=abi.pack(values["gate"], values["up"], values["down"]))
    else:
        want = four_calls(x, ids, w, values, cfg)
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,tm", [(1, 16), (3, 16), (8, 16), (16, 16), (17, 16), (33, 1), (64, 16)])
def test_small_batches(T, tm, dtype):
    """calls planned inside the first launch and calls that are not, with rows beyond 16 of
    one expert (every token goes to expert 3, some twice)"""
    say(f"[mx4] small {T} {tm} {dtype}")
    cfg = custom(f"small_{T}", T=T, d=328, E=40, K=3, f=200, dtype=dtype, tm=tm, x_std=1.0)
    case = make_case(cfg)
    case.ids[:, 1] = 3
    case.ids[::2, 2] = 3
    if T > 2:
        case.ids[2] = -1
        case.ids[1, 0] = cfg.E
    case.drop_device()
    packed, values = four_bits(case)
    out, _ = abi.forward_mx4(case.d("x"), case.d("ids"), case.d("w"), packed, cfg.E, cfg.f, tm=tm,
                             out_dtype=F32)
    want, tol = reference(case, case.ids, values)
    off = np.abs(ref.f64(out) - want)
    assert (off <= tol).all(), np.max(off / tol)


@pytest.mark.parametrize("name", ["decode_bf16", "small_f16", "skipped_bf16"])
def test_layer_against_the_oracle(name):
    say(f"[mx4] oracle {name}")
    cfg = synth.CONFIGS["decode_bf16"] if name == "decode_bf16" else custom(
        name, T=150, d=328, E=12, K=3, f=200, dtype=name.split("_")[1], x_std=1.0)
    case = make_case(cfg)
    ids = case.ids.copy()
    if name == "skipped_bf16":
        ids[::3, 1] = -1
        ids[7] = -1       # a token without an expert
        ids[8, 0] = 4000  # not an expert
    packed, values = four_bits(case)
    out, _ = abi.forward_mx4(case.d("x"), dev(ids), case.d("w"), packed, cfg.E, cfg.f, tm=cfg.tm,
                             out_dtype=F32)
    want = oracle.ffn(case.x, ids, case.w, host(values["gate"]), host(values["up"]),
                      host(values["down"]), cfg.dtype, round_h=True)
    assert rel_err(host(out), want) <= TOL[cfg.dtype]
    if name == "skipped_bf16":
        assert not out[7].any()


def test_a_block_that_is_not_finite_reaches_its_column_only():
    say("[mx4] nan")
    cfg = custom("nan_bf16", T=20, d=64, E=2, K=2, f=40, dtype="bf16", x_std=1.0, w_std=0.2)
    case = make_case(cfg)
    wd = case.d("wd").clone()
    wd[1, 3, 17] = float("nan")
    packed = abi.pack_mx4(case.d("wg"), case.d("wu"), wd)
    out, _ = abi.forward_mx4(case.d("x"), case.d("ids"), case.d("w"), packed, 2, 40, out_dtype=F32)
    bad = out.isnan()
    assert bad[:, 17].all() and bad.sum() == 20


@pytest.mark.parametrize("T,d,E,f", [(131072, 8192, 4, 64), (512, 1 << 21, 32, 8)])
def test_activations_of_2_gib(T, d, E, f):
    """x past what one buffer descriptor addresses: its rows are gathered first, and the
    wide cells (many rows of an expert) or the narrow ones (few) read those. Offsets into
    x, y and the weights pass 32 bits. Of sampled tokens, h is rounded once to fp16
    (2^-11); the sums' roundings are a random walk of at most d / 128 steps of 2^-24 (the
    narrow cells cut d in four), 2^-17 at the most."""
    say(f"[mx4] activations of 2 GiB {T} {d}")
    assert T * d * 2 >= 1 << 31
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, d), generator=g, device="cuda", dtype=F16)
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((T, 1), generator=g, device="cuda") + 0.5
    packed = {}
    for k, kind in (("gate", "gate"), ("up", "gate"), ("down", "down")):
        shape = (E, d, f) if kind == "gate" else (E, f, d)
        m = torch.randn(shape, generator=g, device="cuda", dtype=F16) * shape[1] ** -0.5
        packed[k] = abi.mx4_quantize(m, kind)
        del m
    out, _ = abi.forward_mx4(x, ids, w, packed, E, f, out_dtype=F32)
    toks = [0, 1, T // 2 + 1, T - 2, T - 1]
    rows, eid, wt = x[toks].cpu().double(), ids[toks, 0].tolist(), w[toks, 0].cpu().double()
    got = out[toks].cpu().double()
    del x, out
    values = {k: abi.mx4_dequantize(packed[k], E, d, f, kind, dtype=F16)
              for k, kind in (("gate", "gate"), ("up", "gate"), ("down", "down"))}
    for i, e in enumerate(eid):
        wg, wu, wd = (values[k][e].cpu().double() for k in ("gate", "up", "down"))
        a = rows[i] @ wg
        want = wt[i] * ((a * torch.sigmoid(a) * (rows[i] @ wu)) @ wd)
        assert (got[i] - want).norm() <= 2.0 ** -10 * want.norm(), toks[i]
