"""Plain 64-bit forms of the sequence-mixer operators, token by token on the
CPU, with gradients through autograd (no tests here)."""
import numpy as np
import torch

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of a value near 1, relative
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def spans(B, T, cu):
    if cu is None:
        return [(i, i * T, (i + 1) * T) for i in range(B)]
    return [(n, int(cu[n]), int(cu[n + 1])) for n in range(len(cu) - 1)]


def silu(z):
    return z / (1 + torch.exp(-z))


def conv(x, w, bias, h0, cu, act):
    B, T, D = x.shape
    W = w.shape[1]
    flat = x.reshape(B * T, D)
    ys, hts = [], []
    for n, a, b in spans(B, T, cu):
        old = torch.zeros(W - 1, D, dtype=torch.float64) if h0 is None else h0[n]
        z = torch.cat([old, flat[a:b]])
        pre = sum(z[j:j + b - a] * w[:, j] for j in range(W)) + (0 if bias is None else bias)
        ys.append(silu(pre) if act == "silu" else pre)
        hts.append(z[b - a:])
    return torch.cat(ys).reshape(B, T, D), torch.stack(hts)


def delta_of(dt, dt_bias, softplus):
    z = dt if dt_bias is None else dt + dt_bias
    return torch.logaddexp(z, torch.zeros_like(z)) if softplus else z


def scan(c, b, x, dt, A, D, dt_bias, h0, cu, softplus):
    """A, D, dt_bias: [Hv], or [B, T, Hv] for their gradients token by token."""
    B, T, Hv, V = x.shape
    A = A.expand(B, T, Hv).reshape(B * T, Hv)
    D = None if D is None else D.expand(B, T, Hv).reshape(B * T, Hv)
    Hq, K = c.shape[2:]
    of = torch.arange(Hv) // (Hv // Hq)
    delta = delta_of(dt, dt_bias, softplus).reshape(B * T, Hv)
    c, b, x = c.reshape(B * T, Hq, K)[:, of], b.reshape(B * T, Hq, K)[:, of], x.reshape(B * T, Hv, V)
    ys, hts = [], []
    for n, p, q in spans(B, T, cu):
        S = torch.zeros(Hv, K, V, dtype=torch.float64) if h0 is None else h0[n]
        for t in range(p, q):
            S = torch.exp(delta[t] * A[t])[:, None, None] * S + (delta[t][:, None] * b[t])[:, :, None] * x[t][:, None, :]
            y = (S * c[t][:, :, None]).sum(1)
            ys.append(y if D is None else y + D[t][:, None] * x[t])
        hts.append(S)
    y = torch.stack(ys) if ys else torch.zeros(0, Hv, V, dtype=torch.float64)
    return y.reshape(B, T, Hv, V), torch.stack(hts)


def delta_step(q, k, v, g, beta, S, scale, l2):
    R = v.shape[1] // q.shape[1]
    if l2:
        q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    q, k = q.repeat_interleave(R, 1), k.repeat_interleave(R, 1)
    S = torch.exp(g)[..., None, None] * S
    u = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    return scale * (S * q[..., None]).sum(-2), S


def norm(x, w, b, gate, eps, rms):
    mean = torch.zeros_like(x[..., :1]) if rms else x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    z = (x - mean) * rstd
    z = z if w is None else z * w
    z = z if b is None else z + b
    return z if gate is None else z * silu(gate), mean[..., 0], rstd[..., 0]


def dbl(t):
    return None if t is None else t.detach().cpu().double()


def grads(f, inputs, outs_grads):
    """Gradients of f(*inputs) against outs_grads in 64 bits; None for inputs that are None."""
    leaves = [None if t is None else dbl(t).requires_grad_() for t in inputs]
    pairs = [(y, dbl(d)) for y, d in zip(f(*leaves), outs_grads) if d is not None and y.numel()]
    got = iter(torch.autograd.grad([p[0] for p in pairs], [t for t in leaves if t is not None], [p[1] for p in pairs],
                                   allow_unused=True))
    out = []
    for t in leaves:
        if t is None:
            out.append(None)
            continue
        g = next(got)
        out.append(torch.zeros_like(t) if g is None else g)
    return out


def rel(x, ref):
    x, ref = dbl(x).numpy(), dbl(ref).numpy()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert np.isfinite(x).all()
    n = np.linalg.norm(ref)
    d = np.linalg.norm(x - ref)
    return float(d / n) if n > 0 else float(d)


def near(name, got, ref, tol):
    if ref is None:
        assert got is None, name
        return
    e = rel(got, ref)
    assert e <= tol, f"{name}: {e:.3g} > {tol:.3g}"


def near_sum(name, got, terms, tol):
    """A gradient [Hv] that is a sum over tokens: each term right to tol gives a
    sum that is right to tol times the sum of the terms' sizes (the sum itself
    may cancel to far less)."""
    if terms is None:
        assert got is None, name
        return
    terms = terms.reshape(-1, terms.shape[-1])
    off, most = (dbl(got) - terms.sum(0)).abs(), tol * terms.abs().sum(0)
    assert bool((off <= most).all()), f"{name}: {off.tolist()} > {most.tolist()}"
