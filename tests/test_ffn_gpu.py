"""The gated feed-forward block and its gradients on the GPU, against float64.

Tolerance per element, from the roundings: bf16 operands are exact, products are summed in float32
(K u of the sum over absolute values, u = 2^-24), the activation is within 2^-19 of its size (|g| of
at most 16 or so: an argument's rounding of 2 |g| u and a dozen more), h and the gradients of the
projections are rounded to bf16 (r = 2^-8 relative) and the outputs once more:

  out    |d| <= r |out| + (1 + r) sum |Wd| (r |h| + 2^-19 |h| + e_h),   e_h: g and p off by D u sum |u W|
  grads  from the saved gu, which both sides read: |d| <= r |x| + (1 + r) (r + 2^-18 + K u) sum |A| |B|
"""
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu

U, R = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def ssd():
    import bidirectional_mamba_ssd_bidir_b200 as m
    return m


def _inputs(T, D, F, seed=0):
    g = torch.Generator().manual_seed(zlib.crc32(repr((T, D, F, seed)).encode()))
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = torch.bfloat16
    return r(T, D).to(bf), (r(2 * F, D) / D ** 0.5).to(bf), (r(D, F) / F ** 0.5).to(bf), r(T, D).to(bf)


def _act(name, g):
    """act(g), act'(g) in float64, by the formulas."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * (1 + torch.erf(g / 2 ** 0.5))
    return g * cdf, cdf + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5


def _check(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - tol
    assert bool((over <= 0).all()), f"{what}: off by {(got - ref).abs().max():.3e}, over its bound by {over.max():.3e}"


# tokens: one, a ragged pair of row tiles, more than one tile pair; sizes below, at and past the
# 64 / 128 / 256 steps of the tiles
SIZES = [(1, 8, 8), (1, 256, 512), (3, 64, 136), (17, 200, 1000), (64, 128, 128), (65, 136, 72), (128, 256, 256), (129, 264, 520),
         (200, 512, 1160), (256, 64, 384), (300, 1000, 640), (515, 768, 264), (1000, 24, 2056), (2049, 136, 136),
         (40, 264, 4096), (130, 1032, 2048), (2048, 136, 72)]


@pytest.mark.parametrize("T,D,F", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(ssd, T, D, F, act):
    u, wi, wo, _ = _inputs(T, D, F)
    ws = torch.zeros(ssd.ffn_workspace_bytes(T, D, F), dtype=torch.uint8, device="cuda")
    out, gu = ssd.ffn_block(u.cuda(), wi.cuda(), wo.cuda(), activation=act, save=True, workspace=ws)
    ssd.workspace_status(ws)
    plain = ssd.ffn_block(u.cuda(), wi.cuda(), wo.cuda(), activation=act)
    assert torch.equal(out, plain)                              # saving changes nothing
    u, wi, wo = u.double(), wi.double(), wo.double()
    pre, mag = u @ wi.t(), u.abs() @ wi.abs().t()
    _check(gu, pre, R * pre.abs() + (1 + R) * (D + 8) * U * mag + 1e-30, "gu")
    g, p = pre[:, :F], pre[:, F:]
    a, _ = _act(act, g)
    e = (D + 8) * U
    eh = e * (1.2 * mag[:, :F] * p.abs() + a.abs() * mag[:, F:] + 1.2 * e * mag[:, :F] * mag[:, F:])
    h = a * p
    # GELU far left of zero is a difference (1 + erf): its error is absolute, an ulp of 1
    eh = eh + (U * 8 * g.abs() * p.abs() if act == "gelu" else 0)
    tol = R * (h @ wo.t()).abs() + (1 + R) * ((R + 2.0 ** -19) * h.abs() + eh + F * U * h.abs()) @ wo.abs().t() + 1e-30
    _check(out, h @ wo.t(), tol, "out")


@pytest.mark.parametrize("T,D,F", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(ssd, T, D, F, act):
    u, wi, wo, gy = _inputs(T, D, F, 1)
    gu = (u.float() @ wi.float().t()).to(torch.bfloat16)
    ws = torch.zeros(ssd.ffn_bwd_workspace_bytes(T, D, F), dtype=torch.uint8, device="cuda")
    got = ssd.ffn_block_bwd(u.cuda(), wi.cuda(), wo.cuda(), gu.cuda(), gy.cuda(), activation=act, workspace=ws)
    ssd.workspace_status(ws)
    u, wi, wo, gy, gu = (t.double() for t in (u, wi, wo, gy, gu))
    g, p = gu[:, :F], gu[:, F:]
    a, da = _act(act, g)
    gh, ghm = gy @ wo, (gy.abs() @ wo.abs()) * (D * U)          # ghm: how far gh itself may be off
    ggu = torch.cat([gh * p * da, gh * a], 1)
    # the operands of the three products: value, and how far from it they may be
    slack = torch.cat([ghm * (p * da).abs(), ghm * a.abs()], 1)
    if act == "gelu":
        slack = slack + torch.cat([gh.abs() * p.abs() * 8 * U * (1 + g.abs()), gh.abs() * g.abs() * 8 * U], 1)
    else:                                                       # sigma (1 + g (1 - sigma)) near its zero
        slack = slack + torch.cat([gh.abs() * p.abs() * 16 * U * (1 + g.abs()), 0 * gh], 1)
    off = (R + 2.0 ** -18) * ggu.abs() + (1 + R) * slack
    h = a * p
    hoff = (R + 2.0 ** -18) * h.abs() + (8 * U * (g * p).abs() if act == "gelu" else 0)

    def tol(ref, A, Aoff, B, K):                                # product of A (off by Aoff) and an exact B
        return R * ref.abs() + (1 + R) * (Aoff @ B.abs() + K * U * (A.abs() @ B.abs())) + 1e-30

    ref = ggu @ wi
    _check(got["u"], ref, tol(ref, ggu, off, wi, 2 * F), "u")
    ref = ggu.t() @ u
    _check(got["W_in"], ref, tol(ref, ggu.t(), off.t(), u, T), "W_in")
    ref = (h.t() @ gy).t()
    _check(got["W_out"], ref, tol(ref.t(), h.t(), hoff.t(), gy, T).t(), "W_out")


# ---------------------------------------------------------------- several tiles to a CTA group

def _within(got, ref, tol, what):
    """_check on the GPU."""
    got = got.double()
    assert bool(torch.isfinite(got).all()), what
    over = ((got - ref).abs() - tol).max()
    assert bool(over <= 0), f"{what}: off by {(got - ref).abs().max():.3e}, over its bound by {over:.3e}"


def _tiles(M, N, width, pair):
    """Tiles of the persistent kernel for a product [M][N] (128 or 256 rows, `width` columns), per CTA or pair of them."""
    groups = torch.cuda.get_device_properties(0).multi_processor_count // pair
    return -(-M // (128 * pair)) * -(-N // width) / groups


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_many_tiles_a_group(ssd, act):
    """Accumulators, staging boxes and the load ring handed on from tile to tile, in each launch of the persistent
    kernel: three tiles or more to every CTA pair, ragged in all directions.  Bounds as above; float64 on the GPU."""
    T, D, F = 4100, 3592, 3720
    for M, N, width in ((T, F, 128), (T, D, 256), (T, F, 256), (T, D, 256), (2 * F, D, 256), (D, F, 256)):
        assert _tiles(M, N, width, 2) >= 3
    bf = _inputs(T, D, F, 3)
    u16, wi16, wo16, gy16 = (t.cuda() for t in bf)
    ws = torch.zeros(ssd.ffn_workspace_bytes(T, D, F), dtype=torch.uint8, device="cuda")
    out, gu16 = ssd.ffn_block(u16, wi16, wo16, activation=act, save=True, workspace=ws)
    ssd.workspace_status(ws)
    assert torch.equal(out, ssd.ffn_block(u16, wi16, wo16, activation=act))
    u, wi, wo, gy = (t.double() for t in (u16, wi16, wo16, gy16))
    pre, mag = u @ wi.t(), u.abs() @ wi.abs().t()
    _within(gu16, pre, R * pre.abs() + (1 + R) * (D + 8) * U * mag + 1e-30, "gu")
    g, p = pre[:, :F], pre[:, F:]
    a, _ = _act(act, g)
    h, e = a * p, (D + 8) * U
    eh = e * (1.2 * mag[:, :F] * p.abs() + a.abs() * mag[:, F:] + 1.2 * e * mag[:, :F] * mag[:, F:])
    eh = eh + (U * 8 * g.abs() * p.abs() if act == "gelu" else 0)
    tol = R * (h @ wo.t()).abs() + (1 + R) * ((R + 2.0 ** -19) * h.abs() + eh + F * U * h.abs()) @ wo.abs().t() + 1e-30
    _within(out, h @ wo.t(), tol, "out")
    del pre, mag, eh, tol

    ws = torch.zeros(ssd.ffn_bwd_workspace_bytes(T, D, F), dtype=torch.uint8, device="cuda")
    got = ssd.ffn_block_bwd(u16, wi16, wo16, gu16, gy16, activation=act, workspace=ws)
    ssd.workspace_status(ws)
    g, p = gu16.double().chunk(2, 1)
    a, da = _act(act, g)
    gh, ghm = gy @ wo, (gy.abs() @ wo.abs()) * (D * U)
    ggu = torch.cat([gh * p * da, gh * a], 1)
    slack = torch.cat([ghm * (p * da).abs(), ghm * a.abs()], 1)
    if act == "gelu":
        slack += torch.cat([gh.abs() * p.abs() * 8 * U * (1 + g.abs()), gh.abs() * g.abs() * 8 * U], 1)
    else:
        slack += torch.cat([gh.abs() * p.abs() * 16 * U * (1 + g.abs()), 0 * gh], 1)
    off = (R + 2.0 ** -18) * ggu.abs() + (1 + R) * slack
    h = a * p
    hoff = (R + 2.0 ** -18) * h.abs() + (8 * U * (g * p).abs() if act == "gelu" else 0)

    def tol(ref, A, Aoff, B, K):
        return R * ref.abs() + (1 + R) * (Aoff @ B.abs() + K * U * (A.abs() @ B.abs())) + 1e-30

    ref = ggu @ wi
    _within(got["u"], ref, tol(ref, ggu, off, wi, 2 * F), "u")
    ref = ggu.t() @ u
    _within(got["W_in"], ref, tol(ref, ggu.t(), off.t(), u, T), "W_in")
    ref = (h.t() @ gy).t()
    _within(got["W_out"], ref, tol(ref.t(), h.t(), hoff.t(), gy, T).t(), "W_out")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_many_tiles_a_cta(ssd, act):
    """The same for the single-CTA form of the activation's gradient (up to 128 tokens): its outputs are operands of
    the three products, so a tile that is lost or mixed up shows in all of them."""
    T, D, F = 100, 16, 113800
    assert _tiles(T, F, 256, 1) >= 3
    u16, wi16, wo16, gy16 = (t.cuda() for t in _inputs(T, D, F, 4))
    gu16 = (u16.float() @ wi16.float().t()).to(torch.bfloat16)
    got = ssd.ffn_block_bwd(u16, wi16, wo16, gu16, gy16, activation=act)
    u, wi, wo, gy = (t.double() for t in (u16, wi16, wo16, gy16))
    g, p = gu16.double().chunk(2, 1)
    a, da = _act(act, g)
    gh, ghm = gy @ wo, (gy.abs() @ wo.abs()) * (D * U)
    ggu, h = torch.cat([gh * p * da, gh * a], 1), a * p
    # (1 + |g|) 16 u of the factors covers both activations' derivative
    off = (R + 2.0 ** -18) * ggu.abs() + (1 + R) * torch.cat([ghm * (p * da).abs() + gh.abs() * p.abs() * 16 * U * (1 + g.abs()),
                                                            ghm * a.abs() + gh.abs() * g.abs() * 8 * U], 1)
    hoff = (R + 2.0 ** -18) * h.abs() + 8 * U * (g * p).abs()
    for name, A, Aoff, B, K in (("u", ggu, off, wi, 2 * F), ("W_in", ggu.t(), off.t(), u, T), ("W_out", h.t(), hoff.t(), gy, T)):
        ref = A @ B
        tol = R * ref.abs() + (1 + R) * (Aoff @ B.abs() + K * U * (A.abs() @ B.abs())) + 1e-30
        _within(got[name] if name != "W_out" else got[name].t(), ref, tol, name)


def test_repeats_itself(ssd):
    """Equal inputs give equal bits: the split sums are added in a fixed order."""
    for T, D, F in ((3, 512, 1024), (300, 264, 520), (2100, 136, 264)):
        u, wi, wo, gy = (t.cuda() for t in _inputs(T, D, F, 6))
        (a, gu), (b, _) = (ssd.ffn_block(u, wi, wo, save=True) for _ in range(2))
        g, h = (ssd.ffn_block_bwd(u, wi, wo, gu, gy) for _ in range(2))
        assert torch.equal(a, b) and all(torch.equal(g[k], h[k]) for k in g)


def test_gradient_matches_differences(ssd):
    """The gradients against central differences of the block itself, in float64 on the same inputs."""
    T, D, F = 9, 16, 24
    u, wi, wo, gy = _inputs(T, D, F, 2)
    _, gu = ssd.ffn_block(u.cuda(), wi.cuda(), wo.cuda(), save=True)
    got = ssd.ffn_block_bwd(u.cuda(), wi.cuda(), wo.cuda(), gu, gy.cuda())
    u, wi, wo, gy = (t.double() for t in (u, wi, wo, gy))

    def loss(u, wi, wo):
        g, p = (u @ wi.t()).chunk(2, 1)
        return float(((_act("silu", g)[0] * p) @ wo.t() * gy).sum())

    gen = torch.Generator().manual_seed(5)
    for name, args in (("u", (u, wi, wo)), ("W_in", (u, wi, wo)), ("W_out", (u, wi, wo))):
        i = ("u", "W_in", "W_out").index(name)
        for _ in range(3):
            d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
            eps = 1e-5
            plus, minus = list(args), list(args)
            plus[i], minus[i] = args[i] + eps * d, args[i] - eps * d
            want = (loss(*plus) - loss(*minus)) / (2 * eps)
            have = float((got[name].double().cpu() * d).sum())
            # each gradient element is off by at most about 4 bf16 half steps of its terms
            bound = 6 * R * float((got[name].double().cpu().abs() * d.abs()).sum())
            assert abs(have - want) <= bound, (name, have, want, bound)


def test_leading_dimensions_out_and_graph(ssd):
    """[batch, seqlen, d_model] inputs, a caller's out and workspace, a captured call replayed on new inputs."""
    u, wi, wo, _ = (t.cuda() for t in _inputs(2 * 75, 64, 192))
    u3 = u.view(2, 75, 64)
    out = torch.empty_like(u3)
    ws = torch.zeros(ssd.ffn_workspace_bytes(150, 64, 192), dtype=torch.uint8, device="cuda")
    want = ssd.ffn_block(u, wi, wo)
    assert torch.equal(ssd.ffn_block(u3, wi, wo, out=out, workspace=ws).view(150, 64), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ffn_block(u3, wi, wo, out=out, workspace=ws)
    u3.copy_(u3.flip(1).clone())
    graph.replay()
    want = ssd.ffn_block(u3, wi, wo)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [600, 2300])
def test_training_step_replays_in_a_graph(ssd, T):
    """Forward with saved projections and gradients, captured together and replayed on new tokens: both kernels'
    dependent launches inside a graph."""
    u, wi, wo, gy = (t.cuda() for t in _inputs(T, 136, 264, 7))

    def run():
        out, gu = ssd.ffn_block(u, wi, wo, save=True)
        return [out, gu, *ssd.ffn_block_bwd(u, wi, wo, gu, gy).values()]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        u.copy_(u.flip(0).clone() * 0.5)
        gy.copy_(gy.roll(1, 0).clone())
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_nan_stays_in_its_token(ssd):
    for T in (40, 300):
        u, wi, wo, _ = _inputs(T, 64, 128)
        a = ssd.ffn_block(u.cuda(), wi.cuda(), wo.cuda())
        u[7, 3] = float("nan")
        b = ssd.ffn_block(u.cuda(), wi.cuda(), wo.cuda())
        assert bool(b[7].isnan().all())
        keep = torch.arange(T) != 7
        assert torch.equal(a[keep], b[keep])


def test_empty(ssd):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out, gu = ssd.ffn_block(z(0, 16), z(48, 16), z(16, 24), save=True)
    assert out.shape == (0, 16) and gu.shape == (0, 48)
    g = ssd.ffn_block_bwd(z(0, 16), z(48, 16), z(16, 24), gu, z(0, 16))
    assert g["u"].shape == (0, 16) and bool((g["W_in"] == 0).all()) and bool((g["W_out"] == 0).all())
