"""The layer operators in 64 bits, token by token, with the sums of the terms'
absolute values that the tests' error bounds are made of."""
import torch


def f64(t):
    return t.detach().double()


def heads(v, H):
    """[..., G, n] -> [..., H, n]."""
    return v.repeat_interleave(H // v.shape[-2], dim=-2)


def run_tokens(S, M, x, dt, A, B, C, D):
    """The recurrence from state S [H, dim, dstate] over tokens x [n, H, dim] ...; M is the same with absolute
    values.  Returns (y, |y| sums, S, M)."""
    n, H = x.shape[0], x.shape[1]
    ys, ms = [], []
    for t in range(n):
        a = torch.exp(dt[t] * A)[:, None, None]
        Bt, Ct = heads(B[t], H), heads(C[t], H)
        u = (dt[t][:, None] * x[t])[..., None] * Bt[:, None]
        S, M = a * S + u, a * M + u.abs()
        ys.append((S @ Ct[..., None])[..., 0] + D[:, None] * x[t])
        ms.append((M @ Ct.abs()[..., None])[..., 0] + (D[:, None] * x[t]).abs())
    if n == 0:
        return x.clone(), x.clone(), S, M
    return torch.stack(ys), torch.stack(ms), S, M


def prefill(x, dt, A, B, C, cu, state, initial, D):
    """(y, |y| sums, final states, their sums) of packed sequences; initial: slots or None, negative = zero."""
    H, dim, N = x.shape[1], x.shape[2], B.shape[2]
    x, dt, A, B, C = f64(x), f64(dt), f64(A), f64(B), f64(C)
    D = torch.zeros(H, dtype=torch.float64, device=x.device) if D is None else f64(D)
    y, m = torch.zeros_like(x), torch.zeros_like(x)
    fs, fm = [], []
    for s in range(len(cu) - 1):
        S = torch.zeros(H, dim, N, dtype=torch.float64, device=x.device)
        if initial is not None and initial[s] >= 0:
            S = f64(state[initial[s]])
        k = slice(cu[s], cu[s + 1])
        y[k], m[k], S, M = run_tokens(S, S.abs(), x[k], dt[k], A, B[k], C[k], D)
        fs.append(S)
        fm.append(M)
    return y, m, torch.stack(fs), torch.stack(fm)


def silu(z):
    return z * torch.sigmoid(z)


def rms(v, weight, group, eps):
    w = v.unflatten(-1, (-1, group))
    return (w / (w.pow(2).mean(-1, keepdim=True) + eps).sqrt()).flatten(-2) * weight
