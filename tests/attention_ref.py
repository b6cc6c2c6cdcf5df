"""Plain 64-bit forms of linear attention with a decay for each head (token by
token) and of the channels-last group norm (no tests here)."""
import torch

from tests.mixer_ref import silu, spans


def attention(q, k, v, log_decay, h0, cu, scale):
    B, T, Hv, V = v.shape
    Hq, K = q.shape[2:]
    of = torch.arange(Hv) // (Hv // Hq)
    q, k, v = q.reshape(B * T, Hq, K)[:, of], k.reshape(B * T, Hq, K)[:, of], v.reshape(B * T, Hv, V)
    keep = torch.exp(log_decay)[:, None, None]
    os, hts = [], []
    for n, a, b in spans(B, T, cu):
        S = torch.zeros(Hv, K, V, dtype=torch.float64) if h0 is None else h0[n]
        for t in range(a, b):
            S = keep * S + k[t][:, :, None] * v[t][:, None, :]
            os.append(scale * (S * q[t][:, :, None]).sum(1))
        hts.append(S)
    o = torch.stack(os) if os else torch.zeros(0, Hv, V, dtype=torch.float64)
    return o.reshape(B, T, Hv, V), torch.stack(hts)


def step(q, k, v, log_decay, S, scale):
    R = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(R, 1), k.repeat_interleave(R, 1)
    S = torch.exp(log_decay)[:, None, None] * S + k[..., None] * v[..., None, :]
    return scale * (S * q[..., None]).sum(-2), S


def group_norm(x, groups, w, b, gate, act, eps):
    N, C = x.shape[0], x.shape[-1]
    z = x.reshape(N, -1, groups, C // groups)
    mean = z.mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(((z - mean) ** 2).mean((1, 3), keepdim=True) + eps)
    y = ((z - mean) * rstd).reshape(x.shape)
    y = y if w is None else y * w
    y = y if b is None else y + b
    y = silu(y) if act == "silu" else y
    return y if gate is None else y * silu(gate), mean.reshape(N, groups), rstd.reshape(N, groups)
