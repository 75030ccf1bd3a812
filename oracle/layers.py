"""Float64 forms of the layer operators on packed ragged batches (torch, one sequence at a time, on the inputs' device).

Every function also returns what a tolerance needs: the same sums over absolute values.  Nothing here
is shared with the CUDA path.
"""
import torch


def _order(n, direction):
    return range(n) if direction > 0 else range(n - 1, -1, -1)


def silu(v):
    return v / (1 + torch.exp(-v))


def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def conv(x, w, bias, lens, direction=1, act=True, history=None):
    """x [tokens, C], w [C, K]; lens: length per sequence; history: list of [K-1, C] (oldest first) or None.
    Returns y, the pre-activation, sum |w x| + |bias|, and the list of final histories."""
    x, w = x.double(), w.double()
    C, K = w.shape
    b = bias.double() if bias is not None else torch.zeros(C, dtype=torch.float64)
    y, pre, mag, last = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), []
    lo = 0
    for i, n in enumerate(lens):
        rows = x[lo:lo + n] if direction > 0 else x[lo:lo + n].flip(0)
        h = history[i].double() if history is not None and history[i] is not None else torch.zeros(K - 1, C, dtype=torch.float64)
        ext = torch.cat([h, rows], 0)
        for k in range(n):
            t = lo + k if direction > 0 else lo + n - 1 - k
            prod = w.t() * ext[k:k + K]
            pre[t] = b + prod.sum(0)
            mag[t] = b.abs() + prod.abs().sum(0)
        last.append(ext[ext.shape[0] - (K - 1):])
        lo += n
    return (silu(pre) if act else pre.clone()), pre, mag, last


def conv_bwd(x, w, bias, gy, lens, direction=1, act=True):
    """Gradients by the formulas: gx, gw, gb, and each one's sum over absolute values."""
    x, w, gy = x.double(), w.double(), gy.double()
    C, K = w.shape
    _, pre, _, _ = conv(x, w, bias, lens, direction, act)
    sg = 1 / (1 + torch.exp(-pre))
    gs = gy * (sg * (1 + pre * (1 - sg)) if act else torch.ones_like(pre))
    gx, gw, gb = torch.zeros_like(x), torch.zeros(C, K, dtype=torch.float64), torch.zeros(C, dtype=torch.float64)
    mx, mw, mb = torch.zeros_like(x), torch.zeros_like(gw), torch.zeros_like(gb)
    lo = 0
    for n in lens:
        for k in range(n):
            t = lo + k if direction > 0 else lo + n - 1 - k
            gb += gs[t]
            mb += gs[t].abs()
            for j in range(K):
                if k - j >= 0:                      # x of place k - j entered place k with tap K-1-j
                    s = t - direction * j
                    gw[:, K - 1 - j] += gs[t] * x[s]
                    mw[:, K - 1 - j] += (gs[t] * x[s]).abs()
                    gx[s] += w[:, K - 1 - j] * gs[t]
                    mx[s] += (w[:, K - 1 - j] * gs[t]).abs()
        lo += n
    return (gx, gw, gb), (mx, mw, mb)


def scan(x, dt, A, B, C, D, lens, dt_bias=None, direction=1, start=None):
    """x [tokens, H, P], dt [tokens, H], B, C [tokens, G, N]; start: list of [H, P, N] or None.
    Returns y, the same with absolute values throughout, the final states and theirs."""
    x, dt, A, B, C = x.double(), dt.double(), A.double(), B.double(), C.double()
    T, H, P = x.shape
    G, N = B.shape[1:]
    if dt_bias is not None:
        dt = softplus(dt + dt_bias.double())
    d = D.double() if D is not None else torch.zeros(H, dtype=torch.float64, device=x.device)
    Bh, Ch = B.repeat_interleave(H // G, 1), C.repeat_interleave(H // G, 1)
    y, ym, last, lastm = torch.zeros_like(x), torch.zeros_like(x), [], []
    lo = 0
    for i, n in enumerate(lens):
        S = start[i].double().clone() if start is not None and start[i] is not None else torch.zeros(H, P, N, dtype=torch.float64, device=x.device)
        M = S.abs()
        for t in _order(n, direction):
            t += lo
            a = torch.exp(dt[t] * A)[:, None, None]
            S = a * S + (dt[t][:, None] * x[t])[:, :, None] * Bh[t][:, None, :]
            M = a * M + (dt[t][:, None] * x[t]).abs()[:, :, None] * Bh[t].abs()[:, None, :]
            y[t] = torch.einsum("hpn,hn->hp", S, Ch[t]) + d[:, None] * x[t]
            ym[t] = torch.einsum("hpn,hn->hp", M, Ch[t].abs()) + (d[:, None] * x[t]).abs()
        last.append(S)
        lastm.append(M)
        lo += n
    return y, ym, last, lastm


def step(xBC, dt, conv_w, conv_b, dt_bias, A, D, conv_state, ssm_state, G):
    """One row: xBC [C], dt [H], conv_state [K-1, C], ssm_state [H, P, N]; returns y, |y| sums, states."""
    H, P, N = ssm_state.shape
    v, _, mag, hist = conv(xBC[None], conv_w, conv_b, [1], 1, True, [conv_state])
    v = v[0]
    x, B, C = v[:H * P].reshape(1, H, P), v[H * P:H * P + G * N].reshape(1, G, N), v[H * P + G * N:].reshape(1, G, N)
    y, ym, S, Sm = scan(x, dt[None], A, B, C, D, [1], dt_bias, 1, [ssm_state])
    return y[0], ym[0], hist[0], S[0], Sm[0]
