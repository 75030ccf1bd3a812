"""The layer operators on packed ragged batches and single tokens, on the GPU, against float64.

Tolerances, per element, from the arithmetic (u = 2^-24, h = half a rounding step of the output type
relative to the value: 2^-8 for bf16, 2^-24 for float32):

  conv    s is a sum of K products and the bias in float32: |ds| <= (K + 1) u M with M = |b| + sum |w x|.
          SiLU has slope at most 1.1; its factor sigma is computed from one 2^x and one reciprocal
          (each within 2 u, the argument's rounding adds |s| u) and up to three products: within
          (8 + 2 |s|) u.  So |dy| <= h |y| + (2 (K + 1) M + (8 + 2 |s|) |y|) u.
  scan    the recurrence in float32, token by token: each of the n steps before a token rounds the
          state, its decay (2 u and the argument's rounding, at most |dt A| u) and the new term; a
          product with C and a sum over N: |dy| <= h |y| + (6 n + 2 N + 40) u Y with Y the same
          recurrence over absolute values.  The state: (6 n + 40) u S likewise.
"""
import zlib

import pytest
import torch

from oracle import layers as ol

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ssd():
    import bidirectional_mamba_ssd_bidir_b200 as m
    return m


def _gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def _cu(lens, lead=0):
    c = [lead]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _check(got, ref, tol, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() - tol
    assert bool((bad <= 0).all()), f"{what}: worst {(got - ref).abs().max():.3e}, over its bound by {bad.max():.3e}"


# ---------------------------------------------------------------- convolution

LENS = [[1], [2, 3, 1], [7, 0, 64, 1, 65], [0, 0, 130], [200, 1, 1, 1, 63]]
CONV = [(l, C, K, io, d) for l, C, K, io, d in [
    (LENS[0], 8, 4, "bf16", 1), (LENS[1], 40, 4, "bf16", 1), (LENS[2], 520, 4, "bf16", 1), (LENS[3], 36, 3, "f32", -1),
    (LENS[4], 64, 2, "f32", 1), (LENS[4], 64, 4, "bf16", -1), (LENS[2], 13, 4, "bf16", 1), (LENS[2], 13, 3, "f32", -1),
    (LENS[4], 24, 1, "f32", 1), (LENS[2], 24, 8, "bf16", -1), (LENS[4], 17, 6, "f32", 1)]]


def _conv_tol(io, K, y, pre, mag):
    return HALF[io] * y.abs() + (2 * (K + 1) * mag + (8 + 2 * pre.abs()) * y.abs()) * U * (1 + HALF[io]) + 1e-37


@pytest.mark.parametrize("carry", [False, True], ids=["zero", "carry"])
@pytest.mark.parametrize("lens,C,K,io,direction", CONV, ids=str)
def test_conv(ssd, lens, C, K, io, direction, carry):
    g, dt, T, S = _gen(C, K, io, direction, carry), DT[io], sum(lens), len(lens)
    x = torch.randn(T + 5, C, generator=g).to(dt)
    w, b = torch.rand(C, K, generator=g) - 0.5, torch.randn(C, generator=g)
    pool = torch.randn(S + 2, K - 1, C, generator=g).to(dt)
    slots = torch.randperm(S + 2, generator=g)[:S].to(torch.int32)
    cu = _cu(lens)
    hist = [pool[int(s)] for s in slots] if carry else None
    for act in (True, False):
        out = torch.full((T + 5, C), 7.0, dtype=dt, device="cuda")
        p = pool.cuda()
        kw = dict(state_in=p, state_out=p, slots_in=slots.cuda(), slots_out=slots.cuda()) if carry else {}
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        ssd.ssd_conv(x.cuda(), w.cuda(), b.cuda(), cu_seqlens=cu, direction=direction, silu=act, out=out, workspace=ws, **kw)
        ssd.workspace_status(ws)
        y, pre, mag, last = ol.conv(x[:T], w, b, lens, direction, act, hist)
        _check(out[:T], y, _conv_tol(dt, K, y, pre, mag), "y")
        assert bool((out[T:] == 7).all())                       # rows behind the last sequence
        if carry:
            want = pool.clone()
            for i, s in enumerate(slots):
                want[int(s)] = last[i].to(dt)
            assert torch.equal(p.cpu(), want)                   # states are moved, not computed


def test_conv_no_bias_batched_and_strided(ssd):
    """[batch, seqlen, channels], no bias, x a column block of a wider projection, out one too."""
    g = _gen("strided")
    full = torch.randn(2, 70, 96, generator=g).to(torch.bfloat16)
    w = torch.rand(24, 4, generator=g) - 0.5
    dev = full.cuda()
    keep = dev.clone()
    ssd.ssd_conv(dev[:, :, 16:40], w.cuda(), out=dev[:, :, 48:72])
    y, pre, mag, _ = ol.conv(full[:, :, 16:40].reshape(140, 24), w, None, [70, 70])
    _check(dev[:, :, 48:72].reshape(140, 24), y, _conv_tol(torch.bfloat16, 4, y, pre, mag))
    keep[:, :, 48:72] = dev[:, :, 48:72]
    assert torch.equal(keep, dev)
    odd = ssd.ssd_conv(dev[:, :, 1:14], w[:13].cuda())          # odd offset and channel count: the scalar form
    y, pre, mag, _ = ol.conv(full[:, :, 1:14].reshape(140, 13), w[:13], None, [70, 70])
    _check(odd.reshape(140, 13), y, _conv_tol(torch.bfloat16, 4, y, pre, mag))


def test_conv_nan_and_infinity_stay_in_their_channel(ssd):
    x = torch.zeros(40, 16)
    x[3, 5], x[20, 2], x[30, 9] = float("nan"), float("inf"), -float("inf")
    w = torch.full((16, 3), 0.5)
    y = ssd.ssd_conv(x.cuda(), w.cuda(), cu_seqlens=_cu([22, 18])).cpu()
    want = torch.zeros(40, 16)
    want[3:6, 5] = float("nan")
    want[20:22, 2] = float("inf")                               # its sequence ends at row 22
    want[30:33, 9] = float("nan")                               # -inf * sigma(-inf)
    assert torch.equal(torch.nan_to_num(y, nan=9.0), torch.nan_to_num(want, nan=9.0))


@pytest.mark.parametrize("lens,C,K,io,direction", CONV, ids=str)
@pytest.mark.parametrize("act", [True, False], ids=["silu", "linear"])
def test_conv_bwd(ssd, lens, C, K, io, direction, act):
    g, dt, T = _gen("bwd", C, K, io, direction), DT[io], sum(lens)
    x, gy = torch.randn(T + 3, C, generator=g).to(dt), torch.randn(T + 3, C, generator=g).to(dt)
    w, b = torch.rand(C, K, generator=g) - 0.5, torch.randn(C, generator=g)
    got = ssd.ssd_conv_bwd(x.cuda(), w.cuda(), b.cuda(), gy.cuda(), cu_seqlens=_cu(lens), direction=direction, silu=act)
    (gx, gw, gb), (mx, mw, mb) = ol.conv_bwd(x[:T], w, b, gy[:T], lens, direction, act)
    _, pre, mag, _ = ol.conv(x[:T], w, b, lens, direction, act)
    # silu' has slope at most 0.5; sigma's relative error as above, times the factor's size 1 + |s|:
    # each gs is within e = (0.5 * 2 (K + 1) M + (8 + 2 |s|) (1 + |s|) + 4) u of gy's size
    e = float(((K + 1) * mag + (8 + 2 * pre.abs()) * (1 + pre.abs()) + 4).max()) * U if act else 0.0
    size = float(gy.double().abs().max())
    wsum = w.double().abs().sum(1)
    _check(got["x"][:T], gx, HALF[dt] * gx.abs() + (1 + HALF[dt]) * (e * size * wsum + (K + 1) * U * mx) + 1e-37, "gx")
    assert bool((got["x"][T:] == 0).all())
    n = T
    _check(got["w"], gw, e * size * float(x.double().abs().max()) * n + (n + 4) * U * mw + 1e-37, "gw")
    _check(got["bias"], gb, e * size * n + (n + 4) * U * mb + 1e-37, "gb")


def test_conv_bwd_is_repeatable_and_without_bias(ssd):
    g = _gen("repeat")
    x, gy = (torch.randn(900, 64, generator=g).cuda() for _ in range(2))
    w = (torch.rand(64, 4, generator=g) - 0.5).cuda()
    a, b = (ssd.ssd_conv_bwd(x, w, None, gy, cu_seqlens=_cu([500, 400])) for _ in range(2))
    assert a["bias"] is None and torch.equal(a["w"], b["w"]) and torch.equal(a["x"], b["x"])


# ---------------------------------------------------------------- ragged scan

def _scan_inputs(g, T, H, P, N, G, dt, raw):
    packed = torch.randn(T, H * P + 2 * G * N + 8, generator=g)
    packed[:, H * P:] /= N ** 0.5
    packed = packed.to(dt)
    x = packed[:, :H * P].unflatten(1, (H, P))
    B = packed[:, H * P:H * P + G * N].unflatten(1, (G, N))
    C = packed[:, H * P + G * N:H * P + 2 * G * N].unflatten(1, (G, N))
    d = torch.randn(T, H, generator=g)
    d = (d if raw else torch.nn.functional.softplus(d - 3)).to(dt)
    A = -torch.exp(torch.rand(H, generator=g) * 2.77)
    return packed, x, B, C, d, A, torch.rand(H, generator=g), (torch.randn(H, generator=g) - 3 if raw else None)


SCAN = [
    ([1], 2, 16, 16, 1, "f32", 1), ([3, 0, 17], 4, 32, 64, 2, "f32", -1), ([70, 1, 130], 8, 64, 64, 1, "bf16", 1),
    ([33, 64, 65], 2, 64, 16, 2, "bf16", -1), ([200], 1, 16, 128, 1, "f32", 1), ([129, 40], 4, 32, 32, 4, "bf16", 1),
    ([100, 28], 2, 64, 128, 1, "f32", -1), ([90, 38], 3, 64, 32, 1, "f32", 1), ([64, 64], 2, 32, 128, 1, "bf16", 1),
    ([50], 2, 16, 64, 1, "bf16", -1), ([50], 2, 16, 32, 1, "f32", 1), ([50], 2, 32, 16, 1, "f32", 1),
]


def _scan_case(ssd, lens, H, P, N, G, io, direction, raw, carry, tol_y, tol_s, A=None, skip=True):
    g, dt, T, S = _gen(tuple(lens), H, P, N, raw, carry), DT[io], sum(lens), len(lens)
    packed, x, B, C, d, A0, D, bias = _scan_inputs(g, T + 4, H, P, N, G, dt, raw)
    A = A0 if A is None else A
    D = D if skip else None
    dev = packed.cuda()
    xd, Bd, Cd = (dev.as_strided(v.size(), v.stride(), v.storage_offset()) for v in (x, B, C))
    pool = torch.randn(S + 2, H, P, N, generator=g)
    slots = torch.randperm(S + 2, generator=g)[:S].to(torch.int32)
    p = pool.cuda()
    s_in = dict(state_in=p, slots_in=slots.cuda()) if carry else {}
    out = torch.full((T + 4, H, P), 7.0, dtype=dt, device="cuda")
    ws = torch.zeros(max(256, ssd.ragged_workspace_bytes(T + 4, S, H, P, N, G, dt)), dtype=torch.uint8, device="cuda")
    ssd.ssd_scan_ragged(xd, d.cuda(), A.cuda(), Bd, Cd, D.cuda() if skip else None, cu_seqlens=_cu(lens),
                        dt_bias=bias.cuda() if raw else None, direction=direction, state_out=p, slots_out=slots.cuda(), out=out,
                        workspace=ws, **s_in)
    ssd.workspace_status(ws)
    y, ym, last, lastm = ol.scan(x[:T], d[:T], A, B[:T], C[:T], D, lens, bias, direction,
                                 [pool[int(s)] for s in slots] if carry else None)
    n = max(lens)
    assert bool((out[T:] == 7).all())
    got = p.cpu()
    for i, s in enumerate(slots):
        _check(got[int(s)], last[i], tol_s(n, last[i], lastm[i]), f"state {i}")
    for s in set(range(S + 2)) - set(slots.tolist()):
        assert torch.equal(got[s], pool[s])
    _check(out[:T], y, tol_y(n, N, y, ym), "y")


@pytest.mark.parametrize("carry,raw", [(False, False), (True, True)], ids=["zero", "carry"])
@pytest.mark.parametrize("lens,H,P,N,G,io,direction", SCAN, ids=str)
def test_scan_ragged(ssd, lens, H, P, N, G, io, direction, carry, raw):
    h = HALF[DT[io]]
    _scan_case(ssd, lens, H, P, N, G, io, direction, raw, carry,
               lambda n, N, y, ym: h * y.abs() + (1 + h) * (6 * n + 2 * N + 40) * U * ym + 1e-37,
               lambda n, s, sm: (6 * n + 40) * U * sm + 1e-37)


def test_scan_ragged_pieces_equal_the_whole(ssd):
    """A sequence scanned in ragged pieces, states passed on in slots, against the whole: same recurrence."""
    g = _gen("pieces")
    T, H, P, N = 210, 4, 32, 32
    _, x, B, C, d, A, D, _ = _scan_inputs(g, T, H, P, N, 1, torch.float32, False)
    x, B, C = (v.contiguous().cuda() for v in (x, B, C))
    d, A, D = d.cuda(), A.cuda(), D.cuda()
    whole = torch.zeros(1, H, P, N, device="cuda")
    y = ssd.ssd_scan_ragged(x, d, A, B, C, D, cu_seqlens=_cu([T]), state_out=whole)
    pool = torch.zeros(1, H, P, N, device="cuda")
    parts, lo = [], 0
    for n in (1, 63, 64, 0, 81, 1):
        parts.append(ssd.ssd_scan_ragged(x[lo:lo + n], d[lo:lo + n], A, B[lo:lo + n], C[lo:lo + n], D, cu_seqlens=_cu([n]),
                                         state_in=pool, state_out=pool))
        lo += n
    y64, ym, last, lastm = ol.scan(x.cpu(), d.cpu(), A.cpu(), B.cpu(), C.cpu(), D.cpu(), [T])
    tol = (6 * T + 2 * N + 40) * U
    _check(y, y64, tol * ym)
    _check(torch.cat(parts), y64, tol * ym)
    for s in (whole, pool):
        _check(s[0], last[0], tol * lastm[0])


# The tensor-core form (bf16, headdim 64, d_state 128, pairs of heads).  Within a chunk, a term of y is a
# score rounded to bf16 (2^-8) times a w x rounded to bf16 (2^-8), or in the long form a P rounded once;
# S is rounded to bf16 where it meets C (2^-8); y is rounded (2^-8).  With Y the recurrence over
# absolute values: |dy| <= 2^-8 |y| + (1 + 2^-8) (2 2^-8 + 2^-16 + 2^-12) Y, 2^-12 being room for exponents (|cs|
# up to 500: 500 u ln 2 times a few) and float32 sums.
# The state: w x in three bf16 terms is within 2^-24 (each term leaves at most half a step, 2^-8, of what
# it stands for), B exact; w is within (|cs| + 8) 2 u, |cs| up to 500, sums and decays of n / 128 chunks
# some 3 u each: 2^-14 S.
TC = [
    ([1], 2, 1, 1), ([128], 2, 1, 1), ([127, 129], 4, 2, -1), ([5, 0, 300, 64], 4, 1, 1), ([5, 0, 300, 64], 4, 1, -1),
    ([700], 2, 1, 1), ([513, 130], 2, 1, -1), ([256, 384], 8, 4, 1), ([1] * 9, 2, 1, 1),
]


def _tc_y(n, N, y, ym):
    return 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * (2.0 ** -7 + 2.0 ** -16 + 2.0 ** -12) * ym + 1e-37


def _tc_s(n, s, sm):
    return 2.0 ** -14 * sm + 1e-37


@pytest.mark.parametrize("carry,raw", [(False, False), (True, True)], ids=["zero", "carry"])
@pytest.mark.parametrize("lens,H,G,direction", TC, ids=str)
def test_scan_ragged_tensor_core(ssd, lens, H, G, direction, carry, raw):
    _scan_case(ssd, lens, H, 64, 128, G, "bf16", direction, raw, carry, _tc_y, _tc_s)
    _scan_case(ssd, lens, H, 64, 128, G, "bf16", direction, raw, carry, _tc_y, _tc_s, skip=False)


@pytest.mark.parametrize("direction", [1, -1])
def test_scan_ragged_tensor_core_steep_and_flat(ssd, direction):
    """Decays from none at all (A = 0) to hundreds of powers of two within a chunk."""
    A = torch.tensor([0.0, -0.001, -30.0, -400.0])
    _scan_case(ssd, [300, 77], 4, 64, 128, 1, "bf16", direction, False, True, _tc_y, _tc_s, A=A)


# Several chunks to a segment, several segments to a sequence, with states kept between them: enough heads and
# tokens that a segment is 2 to 7 chunks of 128 (the more heads, the longer the segments).
LONG = [([3000], 64, 1, 1, True), ([1500, 700, 811], 64, 1, -1, False), ([2600, 1, 399], 64, 2, 1, True), ([7003], 64, 4, 1, False),
        ([2304, 2304], 32, 1, -1, True)]


@pytest.mark.parametrize("steep", [1.0, 8.0], ids=["flat", "steep"])
@pytest.mark.parametrize("lens,H,G,direction,carry", LONG, ids=str)
def test_scan_ragged_tensor_core_long(ssd, lens, H, G, direction, carry, steep):
    """As above on long sequences, float64 on the GPU; `steep` sends part of the heads through the long form
    (alternating with the short one from chunk to chunk)."""
    P, N, T, S = 64, 128, sum(lens), len(lens)
    g = _gen(tuple(lens), H, steep)
    _, x, B, C, d, A, D, _ = _scan_inputs(g, T, H, P, N, G, torch.bfloat16, False)
    # stretches of larger steps, so that the chunks of one head differ
    d = (d.float() * (1 + (steep - 1) * (torch.arange(T) // 300 % 3 == 1).float()[:, None])).to(torch.bfloat16)
    x, B, C, d, A, D = (v.contiguous().cuda() for v in (x, B, C, d, A, D))
    pool = torch.randn(S, H, P, N, generator=g).cuda()
    start = [pool[i].clone() for i in range(S)] if carry else None
    ws = torch.zeros(ssd.ragged_workspace_bytes(T, S, H, P, N, G), dtype=torch.uint8, device="cuda")
    y = ssd.ssd_scan_ragged(x, d, A, B, C, D, cu_seqlens=_cu(lens), direction=direction, state_in=pool if carry else None,
                            state_out=pool, workspace=ws)
    ssd.workspace_status(ws)
    ref, ym, last, lastm = ol.scan(x, d, A, B, C, D, lens, None, direction, start)
    _check(y, ref.cpu(), _tc_y(max(lens), N, ref.cpu(), ym.cpu()), "y")
    for i in range(S):
        _check(pool[i], last[i].cpu(), _tc_s(lens[i], last[i].cpu(), lastm[i].cpu()), f"state {i}")


# The states of gently decaying inputs.  With u = 2^-24 and decays of at most 1 (as log2) a chunk: w is one product, one
# ex2 within 4 u and an exponent off by a few u, its product with x and the three terms another 2 u; a chunk's sum of
# 24 steps of the tensor core rounds to some sqrt(24) u in the root mean square, a chunk's decay to 5 u, and two or
# three chunks are remembered: in all some 16 u = 1e-6 relative, as a root mean square over a head's state.  Two
# bf16 terms of w x instead of three would be off by more (tests/test_layers.py measures it on the CPU).
STATE_RMS = 1e-6


@pytest.mark.parametrize("lens,H,direction", [([128], 4, 1), ([900], 64, -1), ([3000], 64, 1), ([1500, 77, 811], 64, -1)], ids=str)
@pytest.mark.parametrize("beside", [0.01, 90.0], ids=["short", "long"])
def test_scan_ragged_tensor_core_states_are_float32(ssd, lens, H, direction, beside):
    """Root mean square error of each gentle head's state.  The other head of a pair decays gently too, or by so much
    that both take the long form; one segment or several, so both kernels that form states are behind it."""
    P, N, T, S = 64, 128, sum(lens), len(lens)
    g = _gen("rms", tuple(lens))
    _, x, B, C, d, _, D, _ = _scan_inputs(g, T, H, P, N, 1, torch.bfloat16, False)
    A = torch.rand(H, generator=g) * -0.04 - 0.01
    A[1::2] = -beside
    x, B, C, d, A, D = (v.contiguous().cuda() for v in (x, B, C, d, A, D))
    pool = torch.empty(S, H, P, N, device="cuda")
    decay = (d.double() * A.double()).abs() / 0.6931
    assert float(decay[:, 0::2].mean()) * 128 < 1 and (beside < 1 or float(decay[:, 1].mean()) * 128 > 300)
    ssd.ssd_scan_ragged(x, d, A, B, C, D, cu_seqlens=_cu(lens), direction=direction, state_out=pool)
    _, _, last, _ = ol.scan(x, d, A, B, C, D, lens, None, direction)
    for i in range(S):
        rms = ((pool[i].double() - last[i]).norm(dim=(1, 2)) / last[i].norm(dim=(1, 2)))[0::2]
        assert float(rms.max()) <= STATE_RMS, (i, rms.max())


@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 44], ids=["small", "large"])
@pytest.mark.parametrize("direction", [1, -1])
def test_scan_ragged_tensor_core_range(ssd, direction, scale):
    """Chunks that decay by just under 2^150, where terms are carried times up to 2^+-76: inputs and states that are
    that much smaller or larger than one keep their bounds (terms up to 2^51 in all; what is below 2^-50 is lost, 128
    such terms are 2^-43, here 2^-13 of the smallest sums)."""
    P, N, H, lens = 64, 128, 4, [300, 77, 128]
    T, S = sum(lens), len(lens)
    g = _gen("range", direction)
    _, x, B, C, _, _, D, _ = _scan_inputs(g, T, H, P, N, 1, torch.bfloat16, False)
    d = torch.full((T, H), 0.0625).to(torch.bfloat16)
    A = torch.tensor([-12.9, -12.5, -12.0, -11.0])              # 128 * 0.0625 * 12.9 / ln 2 = 148.9
    x = (x.float() * scale).to(torch.bfloat16)
    x, B, C, d, A, D = (v.contiguous().cuda() for v in (x, B, C, d, A, D))
    pool = (torch.randn(S, H, P, N, generator=g) * scale).cuda()
    start = [pool[i].clone() for i in range(S)]
    y = ssd.ssd_scan_ragged(x, d, A, B, C, D, cu_seqlens=_cu(lens), direction=direction, state_in=pool, state_out=pool)
    ref, ym, last, lastm = ol.scan(x, d, A, B, C, D, lens, None, direction, start)
    assert float(ym.max()) < 2.0 ** 51
    _check(y, ref.cpu(), _tc_y(T, N, ref.cpu(), ym.cpu()), "y")
    for i in range(S):
        _check(pool[i], last[i].cpu(), _tc_s(T, last[i].cpu(), lastm[i].cpu()), f"state {i}")


@pytest.mark.parametrize("direction", [1, -1])
def test_rows_before_the_first_sequence(ssd, direction):
    """cu_seqlens that does not begin at 0: the rows in front, NaN here, are neither used nor written (zero in gx)."""
    g, lead, tail, lens = _gen("lead", direction), 150, 3, [300, 0, 41]
    n, T = sum(lens), sum(lens) + lead + tail
    inner = slice(lead, lead + n)
    nan = lambda *s: torch.full(s, float("nan"))  # noqa: E731

    def padded(t):
        return torch.cat([nan(lead, *t.shape[1:]), t.float(), nan(tail, *t.shape[1:])]).to(t.dtype).cuda()

    for dt, C in ((torch.bfloat16, 40), (torch.float32, 13)):
        x, gy = torch.randn(n, C, generator=g).to(dt), torch.randn(n, C, generator=g).to(dt)
        w, b = (torch.rand(C, 4, generator=g) - 0.5).cuda(), torch.randn(C, generator=g).cuda()
        out = torch.full((T, C), 7.0, dtype=dt, device="cuda")
        ssd.ssd_conv(padded(x), w, b, cu_seqlens=_cu(lens, lead), direction=direction, out=out)
        assert torch.equal(out[inner], ssd.ssd_conv(x.cuda(), w, b, cu_seqlens=_cu(lens), direction=direction))
        assert bool((out[:lead] == 7).all()) and bool((out[lead + n:] == 7).all())
        a = ssd.ssd_conv_bwd(padded(x), w, b, padded(gy), cu_seqlens=_cu(lens, lead), direction=direction)
        c = ssd.ssd_conv_bwd(x.cuda(), w, b, gy.cuda(), cu_seqlens=_cu(lens), direction=direction)
        assert torch.equal(a["x"][inner], c["x"]) and bool((a["x"][:lead] == 0).all()) and bool((a["x"][lead + n:] == 0).all())
        for k in ("w", "bias"):                                 # the runs begin at other rows: another order of n sums
            assert (a[k] - c[k]).abs().max() <= 4 * n * U * n * 16
    for dt, H, P, N in ((torch.bfloat16, 2, 64, 128), (torch.float32, 2, 32, 16)):
        _, x, B, C, d, A, D, _ = _scan_inputs(g, n, H, P, N, 1, dt, False)
        out = torch.full((T, H, P), 7.0, dtype=dt, device="cuda")
        state = torch.empty(3, H, P, N, device="cuda")
        ssd.ssd_scan_ragged(*(padded(t) for t in (x, d)), A.cuda(), *(padded(t) for t in (B, C)), D.cuda(), cu_seqlens=_cu(lens, lead),
                            direction=direction, state_out=state, out=out)
        ref, ym, last, lastm = ol.scan(x, d, A, B, C, D, lens, None, direction)
        assert bool((out[:lead] == 7).all()) and bool((out[lead + n:] == 7).all())
        if dt is torch.bfloat16:
            ty, ts = _tc_y(300, N, ref, ym), _tc_s
        else:
            ty, ts = (HALF[dt] * ref.abs() + (6 * 300 + 2 * N + 41) * U * ym + 1e-37), lambda k, s, m: (6 * 300 + 40) * U * m + 1e-37  # noqa: E731
        _check(out[inner], ref, ty, "y")
        for i in range(3):
            _check(state[i], last[i], ts(300, last[i], lastm[i]), f"state {i}")


def test_scan_ragged_repeats_itself(ssd):
    """Equal inputs give equal bits, whatever order the jobs are taken in."""
    g = _gen("repeat scan")
    for lens, H, P, N, dt in (([2000, 3, 700], 64, 64, 128, torch.bfloat16), ([300, 20], 4, 32, 64, torch.float32)):
        T, S = sum(lens), len(lens)
        _, x, B, C, d, A, D, _ = _scan_inputs(g, T, H, P, N, 1, dt, False)
        x, B, C, d, A, D = (v.contiguous().cuda() for v in (x, B, C, d, A, D))
        states = [torch.zeros(S, H, P, N, device="cuda") for _ in range(4)]
        ys = [ssd.ssd_scan_ragged(x, d, A, B, C, D, cu_seqlens=_cu(lens), state_out=s) for s in states]
        assert all(torch.equal(ys[0], y) for y in ys) and all(torch.equal(states[0], s) for s in states)


@pytest.mark.parametrize("P,N,io,direction", [(64, 128, "bf16", 1), (64, 128, "bf16", -1), (16, 16, "f32", 1)], ids=str)
def test_scan_ragged_many_sequences(ssd, P, N, io, direction):
    """More sequences than are looked at together, most of them empty or a token long, some of several segments."""
    dt, H = (torch.bfloat16 if io == "bf16" else torch.float32), 2
    lens = [(0, 1, 0, 2, 0)[i % 5] for i in range(1100)]
    for i, n in ((0, 300), (31, 129), (32, 400), (511, 1), (700, 513), (1056, 256), (1099, 131)):
        lens[i] = n
    T, S = sum(lens), len(lens)
    g = _gen("many", P, direction)
    _, x, B, C, d, A, D, _ = _scan_inputs(g, T, H, P, N, 1, dt, False)
    x, B, C, d, A, D = (v.contiguous().cuda() for v in (x, B, C, d, A, D))
    pool = torch.randn(S, H, P, N, generator=g).cuda()
    start = [pool[i].clone() for i in range(S)]
    ws = torch.zeros(ssd.ragged_workspace_bytes(T, S, H, P, N, 1, dt), dtype=torch.uint8, device="cuda")
    y = ssd.ssd_scan_ragged(x, d, A, B, C, D, cu_seqlens=_cu(lens), direction=direction, state_in=pool, state_out=pool,
                            workspace=ws)
    ssd.workspace_status(ws)
    ref, ym, last, lastm = ol.scan(x, d, A, B, C, D, lens, None, direction, start)
    ref, ym, last, lastm = ref.cpu(), ym.cpu(), torch.stack(list(last)).cpu(), torch.stack(list(lastm)).cpu()
    if io == "bf16":
        _check(y, ref, _tc_y(max(lens), N, ref, ym), "y")
        _check(pool, last, _tc_s(max(lens), last, lastm), "states")
    else:
        n = max(lens)
        _check(y, ref, HALF[dt] * ref.abs() + (1 + HALF[dt]) * (6 * n + 2 * N + 40) * U * ym + 1e-37, "y")
        _check(pool, last, (6 * n + 40) * U * lastm + 1e-37, "states")


@pytest.mark.parametrize("P,N,io,direction", [(64, 128, "bf16", 1), (64, 128, "bf16", -1), (32, 32, "f32", -1)], ids=str)
def test_scan_ragged_one_workspace_for_all_batches(ssd, P, N, io, direction):
    """A workspace of the largest batch's size through smaller ones; long sequences among hundreds of short ones (the
    first, some that begin anywhere in a segment, neighbours, the last), whose states pass between the launches."""
    dt, H = DT[io], 8
    g = _gen("one workspace", P, direction)
    lens = [(1, 0, 2, 3)[i % 4] for i in range(640)]
    for i, n in ((0, 700), (13, 257), (14, 129), (15, 385), (300, 256), (301, 1000), (639, 131)):
        lens[i] = n
    ws = torch.zeros(ssd.ragged_workspace_bytes(6000, 700, H, P, N, 1, dt), dtype=torch.uint8, device="cuda")
    for lens in (lens, [1185], lens[:16], lens[::-1], [2, 1], [1700, 3]):
        T, S = sum(lens), len(lens)
        _, x, B, C, d, A, D, _ = _scan_inputs(g, T, H, P, N, 1, dt, False)
        x, B, C, d, A, D = (v.contiguous().cuda() for v in (x, B, C, d, A, D))
        pool = torch.randn(S, H, P, N, generator=g).cuda()
        start = [pool[i].clone() for i in range(S)]
        y = ssd.ssd_scan_ragged(x, d, A, B, C, D, cu_seqlens=_cu(lens), direction=direction, state_in=pool, state_out=pool,
                                workspace=ws)
        ssd.workspace_status(ws)
        ref, ym, last, lastm = ol.scan(x, d, A, B, C, D, lens, None, direction, start)
        ref, ym, last, lastm = ref.cpu(), ym.cpu(), torch.stack(list(last)).cpu(), torch.stack(list(lastm)).cpu()
        n = max(lens)
        if io == "bf16":
            _check(y, ref, _tc_y(n, N, ref, ym), "y")
            _check(pool, last, _tc_s(n, last, lastm), "states")
        else:
            _check(y, ref, HALF[dt] * ref.abs() + (1 + HALF[dt]) * (6 * n + 2 * N + 40) * U * ym + 1e-37, "y")
            _check(pool, last, (6 * n + 40) * U * lastm + 1e-37, "states")


def test_scan_ragged_neighbours_do_not_leak(ssd):
    """NaN and infinity in one sequence (and behind the last) leave the others bit for bit, states too."""
    g = _gen("leak")
    T, H, P, N, lens = 420, 2, 64, 128, [100, 150, 100]
    _, x, B, C, d, A, D, _ = _scan_inputs(g, T, H, P, N, 1, torch.bfloat16, False)
    x, B, C, d = (v.contiguous().cuda() for v in (x, B, C, d))
    for direction in (1, -1):
        def run():
            state = torch.zeros(3, H, P, N, device="cuda")
            y = ssd.ssd_scan_ragged(x, d, A.cuda(), B, C, D.cuda(), cu_seqlens=_cu(lens), direction=direction, state_out=state)
            return y.clone(), state
        keep = [v.clone() for v in (x, B, C, d)]
        y0, s0 = run()
        for t, r in ((x, 120), (x, 200), (B, 130), (C, 140), (d, 150), (x, 360), (B, 360), (d, 360)):
            t[r] = float("nan")
        x[240] = float("inf")
        y1, s1 = run()
        for v, k in zip((x, B, C, d), keep):
            v.copy_(k)
        assert torch.equal(y0[:100], y1[:100]) and torch.equal(y0[250:350], y1[250:350])
        assert torch.equal(s0[0], s1[0]) and torch.equal(s0[2], s1[2])
        assert bool(s1[1].isnan().any())


def test_scan_ragged_unaligned_rows_take_the_other_form(ssd):
    """The tensor-core head shape with rows that a tensor map cannot take: same results within both bounds."""
    g = _gen("unaligned")
    T, H = 150, 2
    wide = torch.randn(T, H * 64 + 2 * 128 + 3, generator=g).to(torch.bfloat16)
    x, B, C = wide[:, 1:129].unflatten(1, (H, 64)), wide[:, 129:257].unflatten(1, (1, 128)), wide[:, 257:385].unflatten(1, (1, 128))
    d, A = torch.rand(T, H, generator=g).mul(0.1).to(torch.bfloat16), -torch.ones(H)
    dev = wide.cuda()
    xd, Bd, Cd = (dev.as_strided(v.size(), v.stride(), v.storage_offset()) for v in (x, B, C))
    y = ssd.ssd_scan_ragged(xd, d.cuda(), A.cuda(), Bd, Cd, cu_seqlens=_cu([T]))
    ref, ym, _, _ = ol.scan(x, d, A, B, C, None, [T])
    _check(y, ref, 2.0 ** -8 * ref.abs() + 1.01 * (6 * T + 300) * U * ym)

# ---------------------------------------------------------------- single tokens

STEP = [(1, 3, 8, 64, 128, 1, 4, "bf16"), (5, 7, 4, 32, 64, 2, 3, "f32"), (17, 17, 2, 16, 16, 1, 2, "f32"),
        (3, 9, 2, 64, 32, 1, 1, "bf16"), (2, 2, 6, 32, 128, 3, 8, "bf16"), (4, 5, 3, 64, 16, 1, 4, "f32"),
        (2, 4, 2, 16, 128, 1, 4, "f32"), (2, 4, 2, 64, 64, 1, 4, "bf16"), (2, 4, 2, 16, 32, 2, 4, "bf16"),
        (2, 4, 2, 16, 64, 1, 4, "f32"), (2, 4, 2, 32, 16, 1, 4, "f32"), (2, 4, 2, 32, 32, 1, 4, "f32")]


def _step_inputs(g, R, n, H, P, N, G, K, dt):
    C = H * P + 2 * G * N
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(xBC=r(R, C).to(dt), dt=r(R, H).to(dt), conv_w=torch.rand(C, K, generator=g) - 0.5, conv_b=r(C), dt_bias=r(H) - 3,
                A=-torch.exp(torch.rand(H, generator=g) * 2.77), D=r(H), conv_state=r(n, K - 1, C).to(dt), ssm_state=r(n, H, P, N))


def _step_row(y, S, a, slot, r, G, K, dt):
    """The convolution's outputs v are within e = ((K + 1) M 2 + (8 + 2 |s|)) u, M = |b| + sum |w x|; they enter
    as x, B and C, so y moves by at most 3 e relative to the sums over (|v| + e); 40 roundings more and N of the sum."""
    yr, ym, hist, S64, Sm = ol.step(a["xBC"][r], a["dt"][r], a["conv_w"], a["conv_b"], a["dt_bias"], a["A"], a["D"],
                                    a["conv_state"][slot], a["ssm_state"][slot], G)
    _, pre, mag, _ = ol.conv(a["xBC"][r:r + 1], a["conv_w"], a["conv_b"], [1], 1, True, [a["conv_state"][slot]])
    e = float((2 * (K + 1) * mag + 8 + 2 * pre.abs()).max()) * U
    H, P, N = S64.shape
    big = 1 + float(pre.abs().max())
    h = HALF[dt]
    # absolute: one factor perturbed by e, the others at most `big`
    _check(S, S64, 40 * U * Sm + 3 * e * big, "state")
    _check(y, yr, h * yr.abs() + (1 + h) * ((2 * N + 60) * U * ym + 3 * e * big * (big + N * (float(S64.abs().max()) + big))), "y")
    return hist.to(dt)


@pytest.mark.parametrize("R,n,H,P,N,G,K,io", STEP, ids=str)
def test_step(ssd, R, n, H, P, N, G, K, io):
    g, dt = _gen("step", R, H, P, N, K), DT[io]
    a = _step_inputs(g, R, n, H, P, N, G, K, dt)
    slots = torch.randperm(n, generator=g)[:R].to(torch.int32)
    if R > 2:
        slots[1] = -1                                           # a padding row
    d = {k: v.cuda() for k, v in a.items()}
    out = torch.full((R, H, P), 7.0, dtype=dt, device="cuda")
    ws = torch.zeros(ssd.step_workspace_bytes(R, H, P, N, G, K), dtype=torch.uint8, device="cuda")
    ssd.mamba2_step(**d, slots=slots.cuda(), ngroups=G, out=out, workspace=ws)
    ssd.workspace_status(ws)
    conv, ssm = a["conv_state"].clone(), d["ssm_state"].cpu()
    for r, s in enumerate(slots.tolist()):
        if s < 0:
            assert bool((out[r] == 7).all())
            continue
        conv[s] = _step_row(out[r], ssm[s], a, s, r, G, K, dt)
    assert torch.equal(d["conv_state"].cpu(), conv)
    for s in set(range(n)) - set(slots.tolist()):
        assert torch.equal(ssm[s], a["ssm_state"][s])


@pytest.mark.parametrize("R,n,H,P,N,G,K,io", [s for s in STEP if s[-1] == "f32"], ids=str)
def test_step_rounds_nothing_in_between(ssd, R, n, H, P, N, G, K, io):
    """float32: element by element, so that a rounding to fewer bits anywhere between the inputs and y would show.
    The convolution's output v is within e = (2 (K + 1) M + (8 + 2 |s|) |v|) u, and with S' the new state
    |dS| <= 40 u |S| + d (e_x |B| + |x| e_B),  |dy| <= (2 N + 60) u Y + sum_n (|dS| |C| + |S'| e_C) + |D| e_x."""
    g = _gen("step exact", R, H, P, N, K)
    a = _step_inputs(g, R, n, H, P, N, G, K, torch.float32)
    slots = torch.randperm(n, generator=g)[:R].to(torch.int32)
    d = {k: v.cuda() for k, v in a.items()}
    y = ssd.mamba2_step(**d, slots=slots.cuda(), ngroups=G).cpu()
    ssm = d["ssm_state"].cpu()
    for r, s in enumerate(slots.tolist()):
        yr, ym, _, S, Sm = ol.step(a["xBC"][r], a["dt"][r], a["conv_w"], a["conv_b"], a["dt_bias"], a["A"], a["D"],
                                   a["conv_state"][s], a["ssm_state"][s], G)
        v, pre, mag, _ = ol.conv(a["xBC"][r:r + 1], a["conv_w"], a["conv_b"], [1], 1, True, [a["conv_state"][s]])
        e = ((2 * (K + 1) * mag + (8 + 2 * pre.abs()) * v.abs()) * U)[0]
        heads = lambda t: (t[:H * P].reshape(H, P), t[H * P:H * P + G * N].reshape(G, N).repeat_interleave(H // G, 0),  # noqa: E731
                           t[H * P + G * N:].reshape(G, N).repeat_interleave(H // G, 0))
        (x, B, C), (ex, eB, eC) = heads(v[0].abs()), heads(e)
        dt = ol.softplus(a["dt"][r].double() + a["dt_bias"].double())[:, None, None]
        eS = 40 * U * Sm + 1.01 * dt * (ex[:, :, None] * B[:, None] + x[:, :, None] * eB[:, None])
        _check(ssm[s], S, eS, "state")
        ey = (2 * N + 60) * U * ym + 1.01 * ((eS * C[:, None]).sum(-1) + (S.abs() * eC[:, None]).sum(-1) + a["D"].double().abs()[:, None] * ex)
        assert float((ey / ym).median()) < 2.0 ** -14           # float32's order, far from bf16's 2^-8
        _check(y[r], yr, ey, "y")


def test_step_strided_rows_and_no_optionals(ssd):
    g = _gen("step strided")
    a = _step_inputs(g, 3, 3, 4, 32, 32, 1, 4, torch.bfloat16)
    a.update(conv_b=None, dt_bias=None, D=None)
    wide = torch.randn(3, a["xBC"].shape[1] + 24, generator=g).to(torch.bfloat16).cuda()
    wide[:, 8:-16] = a["xBC"].cuda()
    wide[:, -12:-8] = (a["dt"].float().abs() * 0.1).to(torch.bfloat16).cuda()
    a["dt"] = wide[:, -12:-8].cpu()
    d = {k: v.cuda() if v is not None else None for k, v in a.items()}
    d["xBC"], d["dt"] = wide[:, 8:-16], wide[:, -12:-8]
    y = ssd.mamba2_step(**d)
    ssm = d["ssm_state"].cpu()
    b = dict(a, conv_b=torch.zeros(wide.shape[1] - 24), dt_bias=torch.zeros(4), D=torch.zeros(4))
    for r in range(3):
        _step_row(y[r], ssm[r], b, r, r, 1, 4, torch.bfloat16)


def test_prompt_then_tokens_equal_one_long_prompt(ssd):
    """A decoding run: ragged prompts through ssd_conv and ssd_scan_ragged into slots, then tokens through
    mamba2_step; the same tokens as longer prompts give the same outputs and states."""
    g = _gen("run")
    H, P, N, G, K, lens, more = 4, 32, 64, 1, 4, [37, 5, 64], 6
    C = H * P + 2 * G * N
    a = _step_inputs(g, 3, 5, H, P, N, G, K, torch.float32)
    w = {k: a[k].cuda() for k in ("conv_w", "conv_b", "dt_bias", "A", "D")}
    xs = [torch.randn(n + more, C, generator=g).cuda() for n in lens]
    ds = [torch.randn(n + more, H, generator=g).cuda() for n in lens]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    none = torch.full((3,), -1, dtype=torch.int32, device="cuda")

    def prompt(x, dt, lens, conv, ssm):
        cu = _cu(lens)
        v = ssd.ssd_conv(x, w["conv_w"], w["conv_b"], cu_seqlens=cu, state_in=conv, state_out=conv, slots_in=none, slots_out=slots)
        return ssd.ssd_scan_ragged(v[:, :H * P].unflatten(1, (H, P)), dt, w["A"], v[:, H * P:H * P + N].unflatten(1, (1, N)),
                                   v[:, H * P + N:].unflatten(1, (1, N)), w["D"], cu_seqlens=cu, dt_bias=w["dt_bias"],
                                   state_in=ssm, state_out=ssm, slots_in=none, slots_out=slots)

    pools = [(torch.randn(5, K - 1, C, generator=g).cuda(), torch.randn(5, H, P, N, generator=g).cuda()) for _ in range(2)]
    whole = prompt(torch.cat(xs), torch.cat(ds), [n + more for n in lens], *pools[0])
    prompt(torch.cat([x[:n] for x, n in zip(xs, lens)]), torch.cat([d[:n] for d, n in zip(ds, lens)]), lens, *pools[1])
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n + more)
    for k in range(more):
        y = ssd.mamba2_step(torch.stack([x[n + k] for x, n in zip(xs, lens)]), torch.stack([d[n + k] for d, n in zip(ds, lens)]),
                            w["conv_w"], w["conv_b"], w["dt_bias"], w["A"], w["D"], *pools[1], slots=slots)
        want = torch.stack([whole[ends[i + 1] - more + k] for i in range(3)])
        assert (y - want).abs().max() <= 1e-5 * want.abs().max()
    used = slots.long()
    assert torch.equal(pools[0][0][used], pools[1][0][used])
    assert (pools[0][1][used] - pools[1][1][used]).abs().max() <= 1e-5 * pools[0][1][used].abs().max()


# ---------------------------------------------------------------- index arrays, graphs, streams

def test_bad_indices_are_reported_and_skipped(ssd):
    """Slots past the pool and slots named twice: the work is skipped, the status word says so."""
    g = _gen("bad")
    a = _step_inputs(g, 3, 4, 2, 16, 16, 1, 4, torch.float32)
    for slots, rows in (([0, 9, 1], [0, 2]), ([2, 3, 2], [1])):
        d = {k: v.cuda() for k, v in a.items()}
        out = torch.full((3, 2, 16), 7.0, device="cuda")
        ws = torch.zeros(ssd.step_workspace_bytes(3, 2, 16, 16), dtype=torch.uint8, device="cuda")
        ssd.mamba2_step(**d, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), out=out, workspace=ws)
        with pytest.raises(ssd.SSDError, match="slot"):
            ssd.workspace_status(ws)
        ssm, conv = d["ssm_state"].cpu(), d["conv_state"].cpu()
        for r in range(3):
            assert bool((out[r] == 7).all()) == (r not in rows)
        done = {slots[r] for r in rows}
        for s in range(4):
            assert torch.equal(ssm[s], a["ssm_state"][s]) == (s not in done)
            assert torch.equal(conv[s], a["conv_state"][s]) == (s not in done)
    x, w = torch.randn(20, 8, generator=g).cuda(), torch.randn(8, 4, generator=g).cuda()
    pool = torch.zeros(3, 3, 8, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for kw, cu in ((dict(state_out=pool, slots_out=i32(1, 1)), _cu([10, 10])), (dict(state_out=pool, slots_out=i32(3, 4)), _cu([10, 10])),
                   (dict(state_in=pool, slots_in=i32(0, 7)), _cu([10, 10])), ({}, i32(0, 15, 10)), ({}, i32(0, 15, 900)),
                   ({}, i32(-4, 15, 20))):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        ssd.ssd_conv(x, w, cu_seqlens=cu, workspace=ws, **kw)
        with pytest.raises(ssd.SSDError, match="slot|cu_seqlens"):
            ssd.workspace_status(ws)
        ssd.workspace_status(ws)                                # cleared by the read
    assert bool((pool == 0).all())
    xs = torch.randn(20, 2, 16, generator=g).cuda()
    B = torch.randn(20, 1, 16, generator=g).cuda()
    d, A = torch.rand(20, 2, generator=g).cuda(), -torch.ones(2, device="cuda")
    ssm = torch.zeros(2, 2, 16, 16, device="cuda")
    for kw, cu in ((dict(state_out=ssm, slots_out=i32(1, 1)), _cu([10, 10])), (dict(state_in=ssm, slots_in=i32(5, 0)), _cu([10, 10])),
                   ({}, i32(0, 18, 12))):
        ws = torch.zeros(ssd.ragged_workspace_bytes(20, 2, 2, 16, 16, 1, torch.float32), dtype=torch.uint8, device="cuda")
        ssd.ssd_scan_ragged(xs, d, A, B, B, cu_seqlens=cu, workspace=ws, **kw)
        with pytest.raises(ssd.SSDError, match="slot|cu_seqlens"):
            ssd.workspace_status(ws)
    assert bool((ssm == 0).all())


def test_a_slot_another_sequence_starts_from_is_kept(ssd):
    """A sequence may end in the slot it started from; a slot that another one starts from is left as it was
    (which of the two came first would be up to the schedule), and the status word says so."""
    g = _gen("kept")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # (slots_in, slots_out, slots that stay as they were)
    cases = [(i32(0, 1), i32(1, 2), [0, 1, 3]), (i32(2, 0), i32(2, 0), [1, 3]), (None, i32(1, 3), [0, 1, 2]),
             (i32(1, 2), None, [1, 2, 3])]

    def check(call, start, nbytes):
        for ins, outs, stay in cases:
            pool, ws = start.clone(), torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
            call(state_in=pool, state_out=pool, slots_in=ins, slots_out=outs, workspace=ws)
            assert [s for s in range(4) if torch.equal(pool[s], start[s])] == stay
            if len(stay) == 2:
                ssd.workspace_status(ws)
            else:
                with pytest.raises(ssd.SSDError, match="slot"):
                    ssd.workspace_status(ws)

    x, w = torch.randn(20, 8, generator=g).cuda(), torch.randn(8, 4, generator=g).cuda()
    check(lambda **kw: ssd.ssd_conv(x, w, cu_seqlens=_cu([10, 10]), **kw), torch.randn(4, 3, 8, generator=g).cuda(), 256)
    for dt, P, N, lens in ((torch.float32, 16, 16, [10, 10]), (torch.bfloat16, 64, 128, [130, 10])):
        T = sum(lens)
        xs, B = torch.randn(T, 2, P, generator=g).to(dt).cuda(), torch.randn(T, 1, N, generator=g).to(dt).cuda()
        d, A = torch.rand(T, 2, generator=g).to(dt).cuda(), -torch.ones(2, device="cuda")
        check(lambda **kw: ssd.ssd_scan_ragged(xs, d, A, B, B, cu_seqlens=_cu(lens), **kw),
              torch.randn(4, 2, P, N, generator=g).cuda(), ssd.ragged_workspace_bytes(T, 2, 2, P, N, 1, dt))


def test_an_out_over_a_state_is_refused(ssd):
    """Refused before anything is launched: the outputs' buffer is a part of the state pool."""
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    conv, ssm = z(2, 3, 8), z(2, 2, 16, 16)
    with pytest.raises(ValueError, match="overlaps a state"):
        ssd.ssd_conv(z(6, 8), z(8, 4), cu_seqlens=_cu([6]), state_out=conv, out=conv.view(6, 8))
    with pytest.raises(ValueError, match="overlaps a state"):
        ssd.ssd_scan_ragged(z(4, 2, 16), z(4, 2), z(2), z(4, 1, 16), z(4, 1, 16), cu_seqlens=_cu([4]), state_in=ssm,
                            out=ssm.view(-1)[:128].view(4, 2, 16))
    conv = z(2, 3, 64)
    for over in (ssm.view(-1)[64:128], conv.view(-1)[:64]):
        with pytest.raises(ValueError, match="overlaps a state"):
            ssd.mamba2_step(z(2, 64), z(2, 2), z(64, 4), None, None, z(2), None, conv, ssm, out=over.view(2, 2, 16))


def test_graph_replays_follow_new_inputs(ssd):
    """A captured decoding step (padded batch, slots in a device tensor) replayed on new contents, and on a
    side stream."""
    g = _gen("graph")
    a = _step_inputs(g, 4, 6, 4, 32, 32, 1, 4, torch.bfloat16)
    d = {k: v.cuda() for k, v in a.items()}
    slots = torch.tensor([1, 3, -1, -1], dtype=torch.int32, device="cuda")
    out = torch.zeros(4, 4, 32, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(ssd.step_workspace_bytes(4, 4, 32, 32), dtype=torch.uint8, device="cuda")
    eager = {k: v.clone() for k, v in d.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ssd.mamba2_step(**{k: v.clone() for k, v in d.items()}, slots=slots, out=out.clone(), workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.mamba2_step(**d, slots=slots, out=out, workspace=ws)
    for new in ([1, 3, -1, -1], [0, 2, 5, -1], [5, 4, 3, 1]):
        x = torch.randn(4, d["xBC"].shape[1], generator=g).to(torch.bfloat16).cuda()
        d["xBC"].copy_(x)
        slots.copy_(torch.tensor(new, dtype=torch.int32))
        eager["xBC"] = x
        want = ssd.mamba2_step(**eager, slots=slots)
        graph.replay()
        torch.cuda.synchronize()
        live = torch.tensor(new) >= 0
        assert torch.equal(out[live], want[live])
        assert torch.equal(d["ssm_state"], eager["ssm_state"]) and torch.equal(d["conv_state"], eager["conv_state"])


def test_empty_sequences_pass_their_states_on(ssd):
    """No token at all (uniform and packed), no sequence at all: states move from slot to slot, gradients are zero."""
    g = _gen("empty")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    conv, ssm = torch.randn(4, 3, 8, generator=g).cuda(), torch.randn(4, 2, 16, 16, generator=g).cuda()
    w = torch.randn(8, 4, generator=g).cuda()
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    kw = dict(slots_in=i32(0, -1), slots_out=i32(3, 2))
    keep_c, keep_s = conv.clone(), ssm.clone()
    ssd.ssd_conv(z(0, 8), w, cu_seqlens=i32(0, 0, 0), state_in=conv, state_out=conv, **kw)
    ssd.ssd_scan_ragged(z(0, 2, 16), z(0, 2), -z(2), z(0, 1, 16), z(0, 1, 16), cu_seqlens=i32(0, 0, 0), state_in=ssm, state_out=ssm, **kw)
    for new, old in ((conv, keep_c), (ssm, keep_s)):
        assert torch.equal(new[3], old[0]) and bool((new[2] == 0).all()) and torch.equal(new[:2], old[:2])
    out = z(2, 3, 16, 16)
    ssd.ssd_scan_ragged(z(2, 0, 3, 16), z(2, 0, 3), -z(3), z(2, 0, 1, 16), z(2, 0, 1, 16), state_out=out.fill_(5))
    assert bool((out == 0).all())
    gr = ssd.ssd_conv_bwd(torch.ones(6, 8, device="cuda"), w, w[:, 0].contiguous(), torch.ones(6, 8, device="cuda"), cu_seqlens=i32(0))
    assert all(bool((gr[k] == 0).all()) for k in ("x", "w", "bias"))


def test_calls_on_a_side_stream_and_two_at_once(ssd):
    """Two scans and two steps on two streams at once, each with its own scratch: as when run alone."""
    g = _gen("streams")
    T, H, P, N = 900, 4, 64, 128
    sets = []
    for i in range(2):
        _, x, B, C, d, A, D, _ = _scan_inputs(g, T, H, P, N, 1, torch.bfloat16, False)
        sets.append([v.contiguous().cuda() for v in (x, d, A, B, C, D)])
    cu = _cu([500, 400])
    alone = [ssd.ssd_scan_ragged(*v, cu_seqlens=cu) for v in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, v in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append([ssd.ssd_scan_ragged(*v, cu_seqlens=cu) for _ in range(4)])
    torch.cuda.synchronize()
    for a, many in zip(alone, got):
        assert all(torch.equal(a, b) for b in many)


def test_conv_and_scan_replay_in_a_graph(ssd):
    """A captured prompt (convolution, then the scan on its column blocks) replayed on new tokens and offsets."""
    g = _gen("graph scan")
    T, H, P, N = 400, 2, 64, 128
    C = H * P + 2 * N
    x = torch.randn(T, C, generator=g).to(torch.bfloat16).cuda()
    d = torch.rand(T, H, generator=g).mul(0.1).to(torch.bfloat16).cuda()
    w, A = (torch.rand(C, 4, generator=g) - 0.5).cuda(), -torch.ones(H, device="cuda")
    cu = _cu([200, 200])
    pool = torch.zeros(2, H, P, N, device="cuda")

    def run():
        v = ssd.ssd_conv(x, w, cu_seqlens=cu)
        return ssd.ssd_scan_ragged(v[:, :H * P].unflatten(1, (H, P)), d, A, v[:, H * P:H * P + N].unflatten(1, (1, N)),
                                   v[:, H * P + N:].unflatten(1, (1, N)), cu_seqlens=cu, state_out=pool)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for lens in ([200, 200], [1, 399], [390, 3]):
        x.copy_(torch.randn(T, C, generator=g))
        cu.copy_(_cu(lens))
        graph.replay()
        got, state = out[:sum(lens)].clone(), pool.clone()
        want = run()
        assert torch.equal(got, want[:sum(lens)]) and torch.equal(state, pool)
