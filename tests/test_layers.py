"""The layer operators without a GPU: host-side refusals of every entry point, and pins of the float64
forms in oracle/layers.py (torch's convolution, differences, the scan oracle).  Nothing here launches a
kernel: every call fails its checks or has nothing to do.
"""
import ctypes

import numpy as np
import pytest
import torch

import bidirectional_mamba_ssd_bidir_b200 as ssd
import oracle
import ssd_inputs as si
from bidirectional_mamba_ssd_bidir_b200 import layers as L
from oracle import layers as ol

GOOD = 1 << 20     # an aligned address that no refused call looks at
OK, INVALID, UNSUPPORTED = 0, 1, 2
lib = ssd.lib


def _err():
    return lib.ssd_last_error().decode()


# ---------------------------------------------------------------- refusals of the C entry points

def _conv(shape=(8, 4, 1, 1, 0), seq=(GOOD, 2, 16), x=GOOD, ldx=8, w=GOOD, b=GOOD, slots=None, y=GOOD, ldy=8, ws=None, wsb=0):
    return lib.ssd_conv(L._ConvShape(*shape), L._Packed(*seq), x, ldx, w, b, L._Slots(*slots) if slots else None, y, ldy, ws, wsb,
                        None)


def test_conv_refusals():
    assert _conv(shape=(0, 4, 1, 1, 0)) == INVALID
    assert _conv(shape=(8, 0, 1, 1, 0)) == UNSUPPORTED and _conv(shape=(8, 9, 1, 1, 0)) == UNSUPPORTED
    assert _conv(shape=(8, 4, 0, 1, 0)) == INVALID and "direction" in _err()
    assert _conv(shape=(8, 4, 1, 1, 7)) == INVALID
    assert _conv(seq=(GOOD, -1, 16)) == INVALID and _conv(seq=(GOOD, 2, -1)) == INVALID
    assert _conv(seq=(None, 3, 16)) == INVALID and "divide" in _err()
    assert _conv(seq=(None, 0, 16)) == INVALID
    assert _conv(seq=(GOOD + 2, 2, 16)) == INVALID
    assert _conv(seq=(GOOD, 1 << 20, 0x7fffffff)) == UNSUPPORTED
    assert _conv(x=None) == INVALID and _conv(x=GOOD + 1) == INVALID and _conv(ldx=7) == INVALID
    assert _conv(y=None) == INVALID and _conv(ldy=7) == INVALID
    assert _conv(w=None) == INVALID and _conv(b=GOOD + 2) == INVALID
    assert _conv(slots=(GOOD + 1, None, None, None, 2, 0)) == INVALID
    assert _conv(slots=(GOOD, None, None, None, 1, 0)) == INVALID and "one slot per sequence" in _err()
    assert _conv(slots=(None, GOOD, None, None, 0, -1)) == INVALID
    assert _conv(ws=GOOD, wsb=255) == INVALID and _conv(ws=GOOD + 2, wsb=256) == INVALID
    assert lib.ssd_conv(None, L._Packed(GOOD, 1, 1), GOOD, 8, GOOD, None, None, GOOD, 8, None, 0, None) == INVALID
    assert lib.ssd_conv(L._ConvShape(8, 4, 1, 1, 0), None, GOOD, 8, GOOD, None, None, GOOD, 8, None, 0, None) == INVALID
    assert _conv(seq=(GOOD, 0, 16), x=None, y=None) == OK            # no sequence: nothing to do


def test_conv_bwd_refusals():
    shape = L._ConvShape(8, 4, 1, 1, 0)
    need = lib.ssd_conv_bwd_workspace_bytes(shape, 300)
    assert need >= 256 + 3 * 5 * 8 * 4
    assert lib.ssd_conv_bwd_workspace_bytes(L._ConvShape(8, 9, 1, 1, 0), 300) == 0
    assert lib.ssd_conv_bwd_workspace_bytes(shape, -1) == 0

    def call(x=GOOD, gy=GOOD, gx=GOOD, gw=GOOD, gb=GOOD, ws=GOOD, wsb=need, ld=8):
        return lib.ssd_conv_bwd(shape, L._Packed(GOOD, 2, 300), x, ld, GOOD, None, gy, ld, gx, ld, gw, gb, ws, wsb, None)

    assert call(gw=None) == INVALID and call(gb=GOOD + 1) == INVALID
    assert call(x=None) == INVALID and call(gy=None) == INVALID and call(gx=None) == INVALID and call(ld=4) == INVALID
    assert call(ws=None) == INVALID and call(ws=GOOD + 16) == INVALID and call(wsb=need - 1) == INVALID


def test_scan_ragged_refusals():
    shape = (4, 32, 64, 2, 1)
    need = lib.ssd_ragged_workspace_bytes(L._RaggedShape(*shape), 100, 3)
    assert need >= 256
    for bad in ((4, 48, 64, 2, 1), (4, 32, 256, 2, 1), (4, 32, 64, 3, 1), (16384, 32, 64, 1, 1), (0, 32, 64, 1, 1), (4, 32, 64, 2, 5)):
        assert lib.ssd_ragged_workspace_bytes(L._RaggedShape(*bad), 100, 3) == 0, bad

    def call(seq=(GOOD, 3, 100), x=GOOD, ldx=128, lddt=4, ldb=128, A=GOOD, D=None, direction=1, slots=None, y=GOOD, ldy=128,
             ws=GOOD, wsb=need, sh=shape):
        p = L._RaggedParams(x, GOOD, GOOD, GOOD, ldx, lddt, ldb, 128, A, D, None)
        return lib.ssd_scan_ragged(L._RaggedShape(*sh), L._Packed(*seq), p, direction, L._Slots(*slots) if slots else None, y, ldy, ws,
                                   wsb, None)

    assert call(x=None) == INVALID and call(ldx=127) == INVALID and call(lddt=3) == INVALID and call(ldb=100) == INVALID
    assert call(A=None) == INVALID and call(D=GOOD + 2) == INVALID and call(direction=2) == INVALID
    assert call(y=None) == INVALID and call(ldy=64) == INVALID
    assert call(ws=None) == INVALID and call(ws=GOOD + 128) == INVALID and call(wsb=need - 1) == INVALID
    assert call(seq=(None, 3, 100)) == INVALID                       # 100 rows in 3 equal sequences
    assert call(slots=(GOOD + 2, None, None, None, 3, 0)) == INVALID and call(slots=(GOOD, None, None, None, 2, 0)) == INVALID
    assert call(sh=(4, 32, 48, 2, 1)) == UNSUPPORTED
    assert call(seq=(GOOD, 0, 100), x=None) == OK


def test_step_refusals():
    shape = (3, 5, 4, 32, 64, 2, 4, 1)
    C = 4 * 32 + 2 * 2 * 64
    need = lib.ssd_step_workspace_bytes(L._StepShape(*shape))
    assert need >= 256 + 3 * C * 4
    for bad in ((-1, 5, 4, 32, 64, 2, 4, 1), (70000, 5, 4, 32, 64, 2, 4, 1), (3, 5, 4, 32, 64, 2, 9, 1), (3, 5, 4, 24, 64, 2, 4, 1)):
        assert lib.ssd_step_workspace_bytes(L._StepShape(*bad)) == 0, bad

    def call(sh=shape, x=GOOD, ldx=C, lddt=4, w=GOOD, A=GOOD, conv=GOOD, ssm=GOOD, slots=GOOD, y=GOOD, ldy=128, ws=GOOD, wsb=need):
        return lib.mamba2_step(L._StepShape(*sh), x, ldx, GOOD, lddt, w, None, None, A, None, conv, ssm, slots, y, ldy, ws, wsb, None)

    assert call(x=None) == INVALID and call(ldx=C - 1) == INVALID and call(lddt=3) == INVALID and call(ldy=127) == INVALID
    assert call(w=None) == INVALID and call(A=None) == INVALID
    assert call(conv=None) == INVALID and call(ssm=None) == INVALID and call(ssm=GOOD + 8) == INVALID
    assert call(slots=GOOD + 2) == INVALID
    assert call(sh=(3, 0, 4, 32, 64, 2, 4, 1)) == INVALID
    assert call(sh=(3, 2, 4, 32, 64, 2, 4, 1), slots=None) == INVALID and "2 slots for 3 rows" in _err()
    assert call(ws=None) == INVALID and call(wsb=need - 1) == INVALID
    assert call(sh=(0, 5, 4, 32, 64, 2, 4, 1), x=None) == OK


def test_ffn_refusals():
    shape = (5, 64, 128, 0)
    fwd, bwd = lib.ssd_ffn_workspace_bytes(L._FfnShape(*shape)), lib.ssd_ffn_bwd_workspace_bytes(L._FfnShape(*shape))
    assert fwd >= 256 + 5 * 128 * 2 and bwd >= 256 + 5 * 3 * 128 * 2
    for bad in ((-1, 64, 128, 0), (5, 60, 128, 0), (5, 64, 100, 0), (5, 0, 128, 0), (5, 64, 128, 2)):
        assert lib.ssd_ffn_workspace_bytes(L._FfnShape(*bad)) == 0, bad

    def call(u=GOOD, wi=GOOD, wo=GOOD, out=GOOD, gu=None, ws=GOOD, wsb=fwd, sh=shape):
        return lib.ffn_block(L._FfnShape(*sh), u, wi, wo, out, gu, ws, wsb, None)

    assert call(u=None) == INVALID and call(wi=GOOD + 8) == INVALID and call(wo=None) == INVALID and call(out=GOOD + 2) == INVALID
    assert call(gu=GOOD + 4) == INVALID and call(ws=None) == INVALID and call(wsb=fwd - 1) == INVALID
    assert call(sh=(5, 60, 128, 0)) == UNSUPPORTED and call(sh=(0, 64, 128, 0), u=None) == OK

    def back(u=GOOD, gu=GOOD, gy=GOOD, g_u=GOOD, gwi=GOOD, gwo=GOOD, wsb=bwd):
        return lib.ffn_block_bwd(L._FfnShape(*shape), u, GOOD, GOOD, gu, gy, g_u, gwi, gwo, GOOD, wsb, None)

    assert back(u=None) == INVALID and back(gu=None) == INVALID and back(gy=GOOD + 8) == INVALID and back(g_u=None) == INVALID
    assert back(gwi=None) == INVALID and back(gwo=GOOD + 4) == INVALID and back(wsb=bwd - 1) == INVALID


def test_pools_that_overlap_in_part_are_refused():
    """A slot that one sequence writes and another reads is told by its number, which overlapping pools would hide."""
    slot = 3 * 8 * 2                                                 # ssd_conv's state here, bytes
    for other in (GOOD + slot, GOOD + 3 * slot + 2, GOOD - 3 * slot, GOOD + 4 * slot - 2):
        assert _conv(slots=(GOOD, other, None, None, 4, 4)) == INVALID and "overlap" in _err()
    need = lib.ssd_ragged_workspace_bytes(L._RaggedShape(4, 32, 64, 2, 1), 100, 3)
    slot = 4 * 32 * 64 * 4
    for other in (GOOD + slot, GOOD - slot, GOOD + 3 * slot - 4):
        p = L._RaggedParams(GOOD, GOOD, GOOD, GOOD, 128, 4, 128, 128, GOOD, None, None)
        assert lib.ssd_scan_ragged(L._RaggedShape(4, 32, 64, 2, 1), L._Packed(GOOD, 3, 100), p, 1,
                                   L._Slots(GOOD, other, None, None, 3, 3), GOOD, 128, GOOD, need, None) == INVALID and "overlap" in _err()
    # the same pool, and two that touch, go on to the checks behind
    for other in (GOOD, GOOD + 4 * 48, GOOD - 4 * 48):
        assert _conv(slots=(GOOD, other, None, None, 4, 4), x=None) == INVALID and "overlap" not in _err()


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    for f in (lambda: ssd.ssd_conv(z(4, 8), z(8, 4), cu_seqlens=z(2, dtype=torch.int32)),
              lambda: ssd.ssd_conv_bwd(z(4, 8), z(8, 4), None, z(4, 8), cu_seqlens=z(2, dtype=torch.int32)),
              lambda: ssd.ssd_scan_ragged(z(1, 4, 2, 16), z(1, 4, 2), z(2), z(1, 4, 1, 16), z(1, 4, 1, 16)),
              lambda: ssd.mamba2_step(z(1, 64), z(1, 2), z(64, 4), None, None, z(2), None, z(1, 3, 64), z(1, 2, 16, 16)),
              lambda: ssd.ffn_block(z(4, 8), z(16, 8), z(8, 8)),
              lambda: ssd.ffn_block_bwd(z(4, 8), z(16, 8), z(8, 8), z(4, 16), z(4, 8))):
        with pytest.raises(ValueError, match="CUDA"):
            f()


class _Dev:
    """The CPU standing in for a device in the checks that come before any call."""
    index = -1


def test_binding_row_checks():
    t = torch.zeros(6, 40)
    rows = lambda v, tail, dtype=torch.float32: L._rows("v", v, False, v.shape[:1], tail, dtype, _Dev)  # noqa: E731
    assert rows(t, (40,)) == (t.data_ptr(), 40)
    assert rows(t[:, 8:24], (16,)) == (t[:, 8:24].data_ptr(), 40)                         # a column block
    assert rows(t[:, 8:24].unflatten(1, (4, 4)), (4, 4)) == (t[:, 8:].data_ptr(), 40)
    dev = t.device
    checked = lambda v, tail, dtype=torch.float32, b=False: L._rows_checked("v", v, b, v.shape[:2 if b else 1], tail, dtype, dev)  # noqa: E731
    with pytest.raises(ValueError, match="contiguous"):
        checked(t[:, ::2], (20,))
    with pytest.raises(ValueError, match="float"):
        checked(t, (40,), torch.bfloat16)
    with pytest.raises(ValueError, match="shape"):
        checked(t, (39,))
    with pytest.raises(ValueError, match="overlap"):
        checked(t.as_strided((5, 8), (4, 1)), (8,))
    assert checked(t.view(2, 3, 40), (40,), b=True) == (t.data_ptr(), 40)
    with pytest.raises(ValueError, match="one behind another"):
        checked(torch.zeros(2, 4, 8)[:, :3], (8,), b=True)


def test_binding_refuses_sizes_past_an_int():
    """2^32 + 5 tokens would reach the C entry points as 5."""
    big, cu = 2 ** 32 + 5, torch.zeros(3, dtype=torch.int32)
    one, w = torch.zeros(1, 1), torch.zeros(8, 8)
    for call in (lambda: L._packed(one.expand(big, 8), 1, cu, _Dev), lambda: L._packed(one.expand(2 ** 16, 2 ** 16)[:, :, None], 1, None, _Dev),
                 lambda: L._packed(torch.zeros(1, 1, 1).expand(big, 0, 8), 1, None, _Dev),
                 lambda: L._ffn_shape(one.expand(big, 8), w, w, "silu", _Dev),
                 lambda: ssd.ragged_workspace_bytes(big, 1, 2, 64, 128), lambda: ssd.ragged_workspace_bytes(1, big, 2, 64, 128),
                 lambda: ssd.step_workspace_bytes(big, 2, 64, 128), lambda: ssd.ffn_workspace_bytes(big, 8, 8),
                 lambda: ssd.ffn_bwd_workspace_bytes(8, big, 8)):
        with pytest.raises(ValueError, match="sizes"):
            call()
    assert L._packed(one.expand(2 ** 31 - 1, 8), 1, cu, _Dev)[0].tokens == 2 ** 31 - 1
    # (the entry points round the tokens up to tiles in ints)
    assert ssd.ffn_workspace_bytes(2 ** 31 - 1, 8, 8) == ssd.ffn_bwd_workspace_bytes(2 ** 31 - 1, 8, 8) == 0


def test_binding_overlap_check():
    t = torch.zeros(6, 40)
    a, b, c = t[:, 0:16], t[:, 16:32], t[:, 10:26]

    def check(out, other):
        L._no_overlap(out, out.data_ptr(), 40, 16, 6, (other, other.data_ptr(), 40, 16))

    check(a, b)
    check(b, a)
    check(a, torch.zeros(6, 40)[:, :16])
    for x, y in ((a, c), (c, a), (b, c), (a, a)):
        with pytest.raises(ValueError, match="overlaps"):
            check(x, y)


def test_binding_refuses_an_out_over_a_state():
    t = torch.zeros(400)
    pool, out = t[:96].view(4, 3, 8), t[96:].view(-1, 16)[:, :8]
    L._apart(out, pool, None)
    L._apart(out, torch.zeros(4, 3, 8))
    L._apart(t[0:0].view(0, 8), pool)
    for o in (t[95:200], t[40:140].view(-1, 20)[:, :8], pool[1], t):
        with pytest.raises(ValueError, match="overlaps a state"):
            L._apart(o, None, pool)


# ---------------------------------------------------------------- pins of the float64 forms

@pytest.mark.parametrize("direction", [1, -1])
@pytest.mark.parametrize("K", [1, 2, 4])
def test_conv_form_is_torchs_convolution(K, direction):
    g = torch.Generator().manual_seed(K)
    lens, C = [5, 1, 9], 6
    x, w, b = torch.randn(15, C, generator=g), torch.randn(C, K, generator=g), torch.randn(C, generator=g)
    hist = [torch.randn(K - 1, C, generator=g) for _ in lens]
    y, _, _, last = ol.conv(x, w, b, lens, direction, True, hist)
    lo = 0
    for i, n in enumerate(lens):
        rows = x[lo:lo + n].double()
        rows = rows if direction > 0 else rows.flip(0)
        ext = torch.cat([hist[i].double(), rows])
        want = torch.nn.functional.silu(torch.nn.functional.conv1d(ext.t()[None], w.double()[:, None], b.double(), groups=C)[0].t())
        assert torch.allclose(y[lo:lo + n], want if direction > 0 else want.flip(0), rtol=0, atol=1e-12)
        assert torch.equal(last[i], ext[n:])
        lo += n


def test_conv_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    lens, C, K = [4, 1, 6], 3, 4
    for direction, act in ((1, True), (-1, True), (1, False)):
        x, w, b, gy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((11, C), (C, K), (C,), (11, C)))
        grads, _ = ol.conv_bwd(x, w, b, gy, lens, direction, act)
        f = lambda x, w, b: float((ol.conv(x, w, b, lens, direction, act)[0] * gy).sum())  # noqa: E731
        for i, v in enumerate((x, w, b)):
            d = torch.randn(v.shape, generator=g, dtype=torch.float64)
            args = [x, w, b]
            up, down = list(args), list(args)
            up[i], down[i] = v + 1e-6 * d, v - 1e-6 * d
            assert abs((f(*up) - f(*down)) / 2e-6 - float((grads[i] * d).sum())) < 1e-7


@pytest.mark.parametrize("direction", [1, -1])
def test_scan_form_is_the_scan_oracle(direction):
    """Equal sequences against the library's scan oracle, which shares nothing with it."""
    shape = si.Shape(3, 20, 4, 16, 16, 2, "f32")
    p, _ = si.make_bidir(shape, seed=4)
    q = oracle.params_f64(p)
    want = oracle.ssd_scan_f64(**q, direction=direction)
    t = {k: torch.from_numpy(np.ascontiguousarray(v)) for k, v in q.items()}
    flat = lambda v: v.reshape(60, *v.shape[2:])  # noqa: E731
    y, _, _, _ = ol.scan(flat(t["x"]), flat(t["dt"]), t["A"], flat(t["B"]), flat(t["C"]), t["D"], [20, 20, 20], None, direction)
    assert np.abs(y.reshape(3, 20, 4, 16).numpy() - want).max() <= 1e-12 * np.abs(want).max()


def test_scan_form_pieces_and_softplus():
    g = torch.Generator().manual_seed(6)
    x, dt, B, C = (torch.randn(*s, generator=g) for s in ((9, 2, 4), (9, 2), (9, 1, 3), (9, 1, 3)))
    A, D, bias = -torch.rand(2, generator=g), torch.rand(2, generator=g), torch.randn(2, generator=g)
    whole, _, last, _ = ol.scan(x, dt, A, B, C, D, [9], bias)
    plain, _, last2, _ = ol.scan(x, torch.nn.functional.softplus(dt.double() + bias.double()), A, B, C, D, [9])
    assert torch.allclose(whole, plain, atol=1e-12) and torch.allclose(last[0], last2[0], atol=1e-12)
    a, _, s, _ = ol.scan(x[:4], dt[:4], A, B[:4], C[:4], D, [4, 0], bias, 1, None)
    b, _, e, _ = ol.scan(x[4:], dt[4:], A, B[4:], C[4:], D, [5], bias, 1, [s[0]])
    assert torch.allclose(torch.cat([a, b]), whole, atol=1e-12) and torch.allclose(e[0], last[0], atol=1e-12)
    assert bool((s[1] == 0).all())                                   # an empty sequence: its start state


def test_three_terms_of_bf16_and_not_two_carry_a_float32_state():
    """What a state built from w x in two or three bf16 terms is off by, as a root mean square: the GPU tests'
    bound for states, 1e-6, lies between the two."""
    g = torch.Generator().manual_seed(8)
    T, P, N = 512, 64, 128
    x, B = (torch.randn(*s, generator=g).to(torch.bfloat16).double() for s in ((T, P), (T, N)))
    w = torch.exp(-torch.rand(T, generator=g)).mul(0.05).double()     # float32 weights
    wx = w[:, None] * x
    exact = wx.t() @ B
    off = []
    for terms in (2, 3):
        left, s = wx.float(), torch.zeros(P, N, dtype=torch.float64)
        for _ in range(terms):
            t = left.to(torch.bfloat16)
            s += t.double().t() @ B
            left = left - t.float()
        off.append(float((s - exact).norm() / exact.norm()))
    assert off[0] > 1.2e-6 and off[1] < 1e-7, off


def test_step_form_is_a_prompt_of_one_token():
    g = torch.Generator().manual_seed(7)
    H, P, N, K = 2, 4, 3, 3
    C = H * P + 2 * N
    xBC, dt, w, b = (torch.randn(*s, generator=g) for s in ((C,), (H,), (C, K), (C,)))
    A, D, bias = -torch.rand(H, generator=g), torch.rand(H, generator=g), torch.randn(H, generator=g)
    conv, ssm = torch.randn(K - 1, C, generator=g), torch.randn(H, P, N, generator=g)
    y, _, hist, S, _ = ol.step(xBC, dt, w, b, bias, A, D, conv, ssm, 1)
    ext = torch.cat([conv, xBC[None]]).double()
    v = torch.nn.functional.silu((ext.t() * w.double()).sum(1) + b.double())
    d = torch.nn.functional.softplus(dt.double() + bias.double())
    want = torch.exp(d * A.double())[:, None, None] * ssm.double() + \
        (d[:, None] * v[:H * P].reshape(H, P))[:, :, None] * v[H * P:H * P + N]
    assert torch.allclose(S, want, atol=1e-12) and torch.equal(hist, ext[1:])
    assert torch.allclose(y, want @ v[H * P + N:] + D.double()[:, None] * v[:H * P].reshape(H, P), atol=1e-12)


def test_ragged_workspace_does_not_fall_as_a_batch_grows():
    """A workspace taken for the largest batch serves every smaller one, in tokens and in sequences."""
    for H, P, N, io in ((64, 64, 128, torch.bfloat16), (2, 64, 128, torch.bfloat16), (600, 64, 128, torch.bfloat16),
                        (8, 32, 64, torch.float32), (700, 16, 16, torch.float32)):
        need = lambda T, S: ssd.ragged_workspace_bytes(T, S, H, P, N, 1, io)  # noqa: E731
        for S in (0, 1, 8, 300):
            sizes = [need(T, S) for T in (*range(0, 2600, 13), *range(2600, 70000, 701))]
            assert sizes == sorted(sizes), (H, S)
        for T in (1, 128, 129, 5000):
            sizes = [need(T, S) for S in range(0, 400, 7)]
            assert sizes == sorted(sizes), (H, T)


def test_ragged_workspace_of_short_sequences():
    """States are kept for sequences of two or more segments alone: at most 2 tokens / segment of them, 38 MB here,
    and 3.3 KB of decay tables a chunk and head."""
    need = lambda T, S: ssd.ragged_workspace_bytes(T, S, 64, 64, 128)  # noqa: E731
    for T, S in ((8192, 4096), (16384, 1024), (16384, 256), (3000, 96)):
        assert need(T, S) <= 39e6 + 64 * (T // 128 + S) * (4 * 840 + 8), (T, S)


def test_workspace_queries_agree_with_the_shapes():
    assert ctypes.sizeof(L._Slots) == 40 and ctypes.sizeof(L._Packed) == 16
    assert ssd.ragged_workspace_bytes(16384, 8, 64, 64, 128) > ssd.ragged_workspace_bytes(100, 1, 64, 64, 128) > 0
    assert ssd.ragged_workspace_bytes(100, 1, 64, 48, 128) == 0
    assert ssd.step_workspace_bytes(4, 64, 64, 128) > 0 and ssd.ffn_workspace_bytes(3, 64, 128) > 0
    assert ssd.ffn_bwd_workspace_bytes(3, 64, 100) == 0
