"""What the sequence-mixer operators around the chunked gated delta rule are measured on.

Operators: the short causal convolution (prompt, backward, single token), the selective state-space
scan (prompt, backward, single token), the single-token gated delta rule, and layer norm with an
optional output gate (forward, backward).  With ``own`` false ``run`` computes them from elementary
torch operations in 32 bits; with ``own`` true it makes the library's calls.

A case is a dict of plain values:
  op      conv_fwd | conv_bwd | conv_step | scan_fwd | scan_bwd | scan_step | delta_step | norm_fwd | norm_bwd
  dtype   bf16 | f32
  B, T    batch rows and tokens each; with N > 0 one packed batch of T tokens cut into N sequences at
          places that ``cut`` (a seed) gives, some of them empty or one token long
  others  sizes and switches of the operator
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


def listed():
    return [
        # prompts of a serving batch, packed: q, k and v channels (H_q = 16, H_v = 32, heads of 128) through the convolution
        {"name": "conv_prompts_bf16", "op": "conv_fwd", "dtype": "bf16", "B": 1, "T": 16384, "N": 16, "cut": 1, "D": 8192, "W": 4,
         "silu": True, "bias": False, "state": True},
        # one training step's backward of the same layer over two rows
        {"name": "conv_train_bf16", "op": "conv_bwd", "dtype": "bf16", "B": 2, "T": 4096, "N": 0, "cut": 0, "D": 8192, "W": 4,
         "silu": True, "bias": True, "state": False},
        # one generated token for each of 32 requests
        {"name": "conv_token_bf16", "op": "conv_step", "dtype": "bf16", "B": 32, "D": 8192, "W": 4, "silu": True, "bias": True,
         "pool": 0, "pad": 0},
        # a long prompt through a state-space layer: 64 heads of 64 over 8 groups, state 128
        {"name": "scan_prompt_bf16", "op": "scan_fwd", "dtype": "bf16", "B": 1, "T": 8192, "N": 0, "cut": 0, "Hq": 8, "Hv": 64,
         "K": 128, "V": 64, "softplus": True, "skip": True, "state": False},
        # a few short prompts of odd lengths that go on from saved states, in full precision
        {"name": "scan_prompts_f32", "op": "scan_fwd", "dtype": "f32", "B": 1, "T": 1277, "N": 7, "cut": 3, "Hq": 2, "Hv": 8,
         "K": 64, "V": 64, "softplus": True, "skip": True, "state": True},
        # one training step's backward over two rows of 4096
        {"name": "scan_train_bf16", "op": "scan_bwd", "dtype": "bf16", "B": 2, "T": 4096, "N": 0, "cut": 0, "Hq": 8, "Hv": 64,
         "K": 128, "V": 64, "softplus": True, "skip": True, "state": False},
        # one generated token for each of 64 requests
        {"name": "scan_token_bf16", "op": "scan_step", "dtype": "bf16", "B": 64, "Hq": 8, "Hv": 64, "K": 128, "V": 64,
         "softplus": True, "skip": True, "pool": 0, "pad": 0},
        # one generated token of one request: latency
        {"name": "delta_token_one_bf16", "op": "delta_step", "dtype": "bf16", "B": 1, "Hq": 16, "Hv": 32, "K": 128, "V": 128,
         "l2norm": True, "pool": 0, "pad": 0},
        # a full decode batch whose states lie in a pool of slots
        {"name": "delta_token_pool_bf16", "op": "delta_step", "dtype": "bf16", "B": 250, "Hq": 16, "Hv": 32, "K": 128, "V": 128,
         "l2norm": True, "pool": 256, "pad": 5},
        # the norm in front of a mixer, a training batch's forward
        {"name": "norm_hidden_bf16", "op": "norm_fwd", "dtype": "bf16", "rows": 16384, "D": 4096, "rms": False, "gate": False,
         "affine": True},
        # the gated norm of the mixer's output heads (8192 tokens, 64 heads of 128), backward
        {"name": "norm_heads_train_bf16", "op": "norm_bwd", "dtype": "bf16", "rows": 524288, "D": 128, "rms": True, "gate": True,
         "affine": True},
        # a wide row with an odd size, backward in full precision
        {"name": "norm_train_f32", "op": "norm_bwd", "dtype": "f32", "rows": 1500, "D": 5003, "rms": False, "gate": False,
         "affine": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "delta_step",
                     "norm_fwd", "norm_bwd"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    packed = rng.random() < 0.5
    if op in ("conv_fwd", "conv_bwd"):
        D = _log(rng, 33, 8192)
        T = _log(rng, 1, min(16384, (1 << 25) // D))
        c |= {"B": 1 if packed else rng.choice([1, 2, 3]), "N": _log(rng, 1, 24) if packed else 0, "cut": rng.randrange(1 << 20),
              "D": D if rng.random() < 0.5 else D // 8 * 8, "W": rng.choice([2, 3, 4]), "silu": rng.random() < 0.7,
              "bias": rng.random() < 0.5, "state": rng.random() < 0.5}
        c["T"] = T if packed else max(1, T // c["B"])
    elif op in ("scan_fwd", "scan_bwd"):
        Hq = rng.choice([1, 2, 4])
        Hv = Hq * rng.choice([1, 2, 3, 4, 8])
        f32 = c["dtype"] == "f32"
        T = _log(rng, 1, 1500 if f32 else 8192)
        c |= {"B": 1 if packed else rng.choice([1, 2, 3]), "N": _log(rng, 1, 16) if packed else 0, "cut": rng.randrange(1 << 20),
              "Hq": Hq, "Hv": Hv, "K": rng.choice([32, 64] if f32 else [32, 64, 128]), "V": rng.choice([32, 64] if f32 else [32, 64, 128]),
              "softplus": rng.random() < 0.8, "skip": rng.random() < 0.7, "state": rng.random() < 0.5}
        c["T"] = T if packed else max(1, T // c["B"])
    elif op == "conv_step":
        c |= {"B": _log(rng, 1, 512), "D": _log(rng, 33, 8192), "W": rng.choice([2, 3, 4]), "silu": rng.random() < 0.7,
              "bias": rng.random() < 0.5}
    elif op in ("scan_step", "delta_step"):
        Hq = _log(rng, 1, 16)
        c |= {"B": _log(rng, 1, 150), "Hq": Hq, "Hv": Hq * rng.choice([1, 2, 3]), "K": rng.choice([32, 64, 128]),
              "V": rng.choice([32, 64, 128])}
        c |= {"l2norm": rng.random() < 0.5} if op == "delta_step" else {"softplus": rng.random() < 0.8, "skip": rng.random() < 0.7}
    else:
        D = _log(rng, 32, 16384)
        c |= {"D": D, "rows": _log(rng, 1, (1 << 25) // D), "rms": rng.random() < 0.5, "gate": rng.random() < 0.5,
              "affine": rng.random() < 0.8}
    if op.endswith("_step"):
        c |= {"pool": c["B"] + rng.randrange(1, 9), "pad": rng.randrange(0, (c["B"] + 1) // 2)} if packed else {"pool": 0, "pad": 0}
    return c


# ---------------------------------------------------------------- inputs


def _cuts(case):
    """Sequence borders of a packed batch: N lengths that add up to T, empty ones and single tokens among them."""
    r = random.Random(case["cut"])
    at = sorted(r.choice([0, r.randrange(case["T"] + 1), r.randrange(case["T"] + 1), min(case["T"], 1)]) for _ in range(case["N"] - 1))
    return [0] + at + [case["T"]]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt, op = DT[case["dtype"]], case["op"]

    def normal(*shape, like=None):
        return torch.randn(*shape, generator=gen, device="cuda").to(dt if like is None else like)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    def act(*shape):  # what a convolution with SiLU in front leaves
        z = torch.randn(*shape, generator=gen, device="cuda")
        return (z * torch.sigmoid(z)).to(dt)

    f32 = torch.float32
    s = {"case": case, "cu": None}
    if case.get("N"):
        s["cuts"] = _cuts(case)
        s["cu"] = torch.tensor(s["cuts"], dtype=torch.int32, device="cuda")
    if op.endswith("_step"):
        slots = case["pool"] or case["B"]
        s["index"] = None
        if case["pool"]:
            s["index"] = torch.randperm(slots, generator=gen, device="cuda")[: case["B"]].to(torch.int32)
            s["index"][case["B"] - case["pad"]:] = -1
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        D, W = case["D"], case["W"]
        s["weight"] = (normal(D, W, like=f32) * W ** -0.5).to(dt)
        s["bias"] = (0.1 * normal(D, like=f32)).to(dt) if case["bias"] else None
        if op == "conv_step":
            s["x"], s["state"] = normal(case["B"], D), normal(slots, W - 1, D)
            return s
        rows = case["N"] or case["B"]
        s["x"] = normal(case["B"], case["T"], D)
        s["h0"] = normal(rows, W - 1, D) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = normal(case["B"], case["T"], D)
            s["dht"] = normal(rows, W - 1, D) if case["state"] else None
        return s
    if op in ("scan_fwd", "scan_bwd", "scan_step"):
        Hq, Hv, K, V = (case[k] for k in ("Hq", "Hv", "K", "V"))
        lead = (case["B"],) if op == "scan_step" else (case["B"], case["T"])
        s["c"], s["b"], s["x"] = act(*lead, Hq, K), act(*lead, Hq, K), act(*lead, Hv, V)
        s["A"] = -uniform(1, 16, Hv)
        s["D"] = 1 + 0.1 * normal(Hv, like=f32) if case["skip"] else None
        step = torch.exp(uniform(-6.9, -2.3, Hv))  # the step sizes 0.001 .. 0.1 that such layers start from
        if case["softplus"]:
            s["dt_bias"] = step + torch.log(-torch.expm1(-step))
            s["dt"] = normal(*lead, Hv)
        else:
            s["dt_bias"] = None
            s["dt"] = (step * torch.exp(0.5 * normal(*lead, Hv, like=f32))).to(dt)
        if op == "scan_step":
            s["state"] = 0.1 * normal(slots, Hv, K, V, like=f32)
            return s
        rows = case["N"] or case["B"]
        s["h0"] = 0.1 * normal(rows, Hv, K, V, like=f32) if case["state"] else None
        if op == "scan_bwd":
            s["dy"] = normal(*lead, Hv, V)
            s["dht"] = 0.1 * normal(rows, Hv, K, V, like=f32) if case["state"] else None
        return s
    if op == "delta_step":
        B, Hq, Hv, K, V = (case[k] for k in ("B", "Hq", "Hv", "K", "V"))
        q, k = normal(B, Hq, K, like=f32), normal(B, Hq, K, like=f32)
        if not case["l2norm"]:
            q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), normal(B, Hv, V)
        z = normal(B, Hv, like=f32)
        s["g"] = -(torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))) / 10
        s["beta"] = torch.sigmoid(normal(B, Hv, like=f32)).to(dt)
        s["state"] = 0.1 * normal(slots, Hv, K, V, like=f32)
        return s
    rows, D = case["rows"], case["D"]
    s["x"] = (normal(rows, D, like=f32) * torch.exp(0.5 * normal(rows, 1, like=f32)) + 0.3).to(dt)
    s["weight"] = 1 + 0.1 * normal(D, like=f32) if case["affine"] else None
    s["bias"] = 0.1 * normal(D, like=f32) if case["affine"] and not case["rms"] else None
    s["gate"] = normal(rows, D) if case["gate"] else None
    if op == "norm_bwd":  # what the forward left
        s["dy"] = normal(rows, D)
        x = s["x"].double()
        s["mean"] = None if case["rms"] else x.mean(-1).float()
        s["rstd"] = ((x * x if case["rms"] else (x - x.mean(-1, keepdim=True)) ** 2).mean(-1) + EPS).rsqrt().float()
    return s


EPS = 1e-5


# ---------------------------------------------------------------- the plain forms


def _f(t):
    return None if t is None else t.float()


def _grad(f, inputs, outs_grads):
    """Gradients of f(*inputs) (a tuple of tensors) against outs_grads; inputs that are None stay None."""
    leaves = [None if t is None else t.detach().float().requires_grad_() for t in inputs]
    with torch.enable_grad():
        pairs = [(y, d) for y, d in zip(f(*leaves), outs_grads) if d is not None]
        got = iter(torch.autograd.grad([p[0] for p in pairs], [t for t in leaves if t is not None], [p[1].float() for p in pairs]))
    return [None if t is None else next(got).to(t.dtype) for t in inputs]


def _silu(z):
    return z * torch.sigmoid(z)


def _where(s, T):
    """For each of B * T tokens in a row: its sequence and the first token of that; and each sequence's end."""
    case, dev = s["case"], "cuda"
    t = torch.arange(T * case["B"], device=dev)
    if s["cu"] is None:
        n = t // T
        return n, n * T, (torch.arange(case["B"], device=dev) + 1) * T
    cu = s["cu"].long()
    n = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return n, cu[n], cu[1:]


def _conv(s, x, weight, bias, h0):
    case = s["case"]
    (B, T, D), W = x.shape, case["W"]
    rows = case["N"] or B
    n, first, ends = _where(s, T)
    old = x.new_zeros(rows, W - 1, D) if h0 is None else h0
    every = torch.cat([x.reshape(B * T, D), old.reshape(rows * (W - 1), D)])

    def at(t, n, first):  # the row of `every` that holds the input at token t of sequence n
        return torch.where(t >= first, t, B * T + n * (W - 1) + (W - 1) + t - first)

    taps = torch.arange(W, device=x.device) - (W - 1)
    src = at(torch.arange(B * T, device=x.device)[:, None] + taps, n[:, None], first[:, None])
    y = (every[src] * weight.t()).sum(1)
    y = y if bias is None else y + bias
    starts = torch.cat([ends.new_zeros(1), ends[:-1]])
    last = at(ends[:, None] + taps[1:] - 1, torch.arange(rows, device=x.device)[:, None], starts[:, None])
    return (_silu(y) if case["silu"] else y).reshape(B, T, D), every[last]


def _softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))


def _scan(s, c, b, x, dt, A, D, dt_bias, h0):
    """Chunks of 64 tokens: products inside a chunk, and the states between chunks from the decays between them."""
    case = s["case"]
    (B, T), (Hq, Hv, K, V) = x.shape[:2], (case[k] for k in ("Hq", "Hv", "K", "V"))
    rows = case["N"] or B
    n_of, first, ends = _where(s, T)
    L = max([q - p for p, q in zip(s["cuts"], s["cuts"][1:])]) if s["cu"] is not None else T
    nc = (L + CHUNK - 1) // CHUNK
    starts = torch.cat([ends.new_zeros(1), ends[:-1]])
    at = starts[:, None] + torch.arange(nc * CHUNK, device=x.device)  # every sequence padded to nc chunks
    live = at < ends[:, None]
    at = torch.clamp(at, max=B * T - 1)

    def cut(t):  # [B, T, H, ..] -> [rows, nc, H, CHUNK, ..]
        t = t.reshape(B * T, *t.shape[2:])[at]
        return t.reshape(rows, nc, CHUNK, *t.shape[2:]).transpose(2, 3)

    zero = dt if dt_bias is None else dt + dt_bias
    delta = cut(_softplus(zero) if case["softplus"] else zero) * live.reshape(rows, nc, 1, CHUNK)
    gam = torch.cumsum((delta * A[:, None]).double(), -1)  # [rows, nc, Hv, CHUNK]
    c, b, x_ = cut(c), cut(b), cut(x)
    R = Hv // Hq
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    E = torch.exp((gam[..., :, None] - gam[..., None, :]).masked_fill(~low, float("-inf"))).float()
    P = (c @ b.transpose(-1, -2)).repeat_interleave(R, 2) * E * delta[..., None, :]
    w = (torch.exp(gam[..., -1:] - gam)).float() * delta
    U = (b.transpose(-1, -2).repeat_interleave(R, 2) * w[..., None, :]) @ x_  # what each chunk adds to the state
    tot = torch.cumsum(gam[..., -1].double(), 1).transpose(1, 2)  # [rows, Hv, nc]
    tot = torch.cat([tot.new_zeros(rows, Hv, 1), tot], -1)
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    W = torch.exp((tot[..., :, None] - tot[..., None, :]).masked_fill(~low, float("-inf"))).float()
    h0 = x.new_zeros(rows, Hv, K, V) if h0 is None else h0
    S = (W @ torch.cat([h0[:, None], U], 1).transpose(1, 2).reshape(rows, Hv, nc + 1, K * V)).reshape(rows, Hv, nc + 1, K, V)
    y = P @ x_ + torch.exp(gam).float()[..., None] * (c.repeat_interleave(R, 2) @ S[:, :, :nc].transpose(1, 2).contiguous())
    y = y.transpose(2, 3).reshape(rows, nc * CHUNK, Hv, V)
    y = y[n_of, torch.arange(B * T, device=x.device) - first].reshape(B, T, Hv, V)
    y = y if D is None else y + D[:, None] * x
    return y, S[:, :, nc]


def _slots(s):
    """The live rows of a step's batch and their slots (the rows behind them are padding)."""
    case = s["case"]
    live = case["B"] - case["pad"]
    return live, slice(0, live) if s["index"] is None else s["index"][:live].long()


def _with_padding(s, y):
    pad = s["case"]["pad"]
    return torch.cat([y, y.new_zeros(pad, *y.shape[1:])]) if pad else y


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DT[case["dtype"]]
    if op == "conv_fwd":
        y, ht = _conv(s, _f(s["x"]), _f(s["weight"]), _f(s["bias"]), _f(s["h0"]))
        return y.to(dt), ht.to(dt)
    if op == "conv_bwd":
        return _grad(lambda *a: _conv(s, *a), [s["x"], s["weight"], s["bias"], s["h0"]], [s["dy"], s["dht"]])
    if op == "conv_step":
        live, at = _slots(s)
        win = torch.cat([s["state"][at].float(), s["x"][:live, None].float()], 1)  # [live, W, D]
        y = (win * s["weight"].float().t()).sum(1)
        y = y if s["bias"] is None else y + s["bias"].float()
        s["state"][at] = win[:, 1:].to(dt)
        return _with_padding(s, (_silu(y) if case["silu"] else y).to(dt)), s["state"]
    if op == "scan_fwd":
        y, ht = _scan(s, *(_f(s[k]) for k in ("c", "b", "x", "dt", "A", "D", "dt_bias", "h0")))
        return y.to(dt), ht
    if op == "scan_bwd":
        return _grad(lambda *a: _scan(s, *a), [s[k] for k in ("c", "b", "x", "dt", "A", "D", "dt_bias", "h0")], [s["dy"], s["dht"]])
    if op == "scan_step":
        live, at = _slots(s)
        R = case["Hv"] // case["Hq"]
        c, b, x, z = (s[k][:live].float() for k in ("c", "b", "x", "dt"))
        z = z if s["dt_bias"] is None else z + s["dt_bias"]
        delta = _softplus(z) if case["softplus"] else z
        S = torch.exp(delta * s["A"])[..., None, None] * s["state"][at]
        S = S + (delta[..., None] * b.repeat_interleave(R, 1))[..., :, None] * x[..., None, :]
        y = (S * c.repeat_interleave(R, 1)[..., :, None]).sum(-2)
        y = y if s["D"] is None else y + s["D"][:, None] * x
        s["state"][at] = S
        return _with_padding(s, y.to(dt)), s["state"]
    if op == "delta_step":
        live, at = _slots(s)
        R = case["Hv"] // case["Hq"]
        q, k, v, beta, g = (s[n][:live].float() for n in ("q", "k", "v", "beta", "g"))
        if case["l2norm"]:
            q, k = (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        q, k = q.repeat_interleave(R, 1)[..., :, None], k.repeat_interleave(R, 1)[..., :, None]
        S = torch.exp(g)[..., None, None] * s["state"][at]
        u = beta[..., None] * (v - (S * k).sum(-2))
        S = S + k * u[..., None, :]
        y = case["K"] ** -0.5 * (S * q).sum(-2)
        s["state"][at] = S
        return _with_padding(s, y.to(dt)), s["state"]

    def norm(x, weight, bias, gate):
        mean = x.new_zeros(x.shape[0], 1) if case["rms"] else x.mean(-1, keepdim=True)
        rstd = torch.rsqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS)
        y = (x - mean) * rstd
        y = y if weight is None else y * weight
        y = y if bias is None else y + bias
        return y if gate is None else y * _silu(gate), mean[:, 0], rstd[:, 0]

    args = [s[k] for k in ("x", "weight", "bias", "gate")]
    if op == "norm_fwd":
        y, mean, rstd = norm(*map(_f, args))
        return y.to(dt), None if case["rms"] else mean, rstd
    return _grad(norm, args, [s["dy"], None, None])


# ---------------------------------------------------------------- the library's calls


def _library(s):
    import gated_deltanet_chunked_gdn_amd as gdn
    case, op = s["case"], s["case"]["op"]
    act = "silu" if case.get("silu") else None
    if op == "conv_fwd":
        return gdn.causal_conv_fwd(s["x"], s["weight"], s["bias"], initial_state=s["h0"], cu_seqlens=s["cu"], activation=act,
                                   check_cu_seqlens=False)
    if op == "conv_bwd":
        return gdn.causal_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], initial_state=s["h0"], dfinal_state=s["dht"],
                                   cu_seqlens=s["cu"], activation=act, check_cu_seqlens=False)
    if op == "conv_step":
        return gdn.causal_conv_step(s["x"], s["state"], s["weight"], s["bias"], activation=act, state_indices=s["index"]), s["state"]
    if op == "scan_fwd":
        return gdn.selective_scan_fwd(s["c"], s["b"], s["x"], s["dt"], s["A"], D=s["D"], dt_bias=s["dt_bias"],
                                      dt_softplus=case["softplus"], initial_state=s["h0"], cu_seqlens=s["cu"], check_cu_seqlens=False)
    if op == "scan_bwd":
        return gdn.selective_scan_bwd(s["c"], s["b"], s["x"], s["dt"], s["A"], s["dy"], dht=s["dht"], D=s["D"], dt_bias=s["dt_bias"],
                                      dt_softplus=case["softplus"], initial_state=s["h0"], cu_seqlens=s["cu"], check_cu_seqlens=False)
    if op == "scan_step":
        return gdn.selective_scan_step(s["c"], s["b"], s["x"], s["dt"], s["A"], s["state"], D=s["D"], dt_bias=s["dt_bias"],
                                       dt_softplus=case["softplus"], state_indices=s["index"]), s["state"]
    if op == "delta_step":
        return gdn.gated_delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"],
                                         use_qk_l2norm_in_kernel=case["l2norm"], state_indices=s["index"]), s["state"]
    if op == "norm_fwd":
        return gdn.layer_norm_fwd(s["x"], s["weight"], s["bias"], gate=s["gate"], eps=EPS, rms=case["rms"])
    return gdn.layer_norm_bwd(s["dy"], s["x"], s["weight"], s["bias"], s["mean"], s["rstd"], gate=s["gate"], rms=case["rms"])


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- sizes


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("conv"):
        n = case["B"] * case.get("T", 1) * case["D"]
        rows = (case["N"] or case["B"]) if "N" in case else case["B"] - case["pad"]
        st = rows * (case["W"] - 1) * case["D"] * e
        if op == "conv_step":
            return {"bytes": 2 * n * e + 2 * st + case["D"] * case["W"] * e, "flops": 2 * n * case["W"]}
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + st * (1 + case["state"]) + case["D"] * case["W"] * e, "flops": 2 * n * case["W"]}
        return {"bytes": 3 * n * e + 3 * st * case["state"] + 2 * case["D"] * case["W"] * e, "flops": 6 * n * case["W"]}
    if op in ("scan_fwd", "scan_bwd", "scan_step", "delta_step"):
        Hq, Hv, K, V = (case[k] for k in ("Hq", "Hv", "K", "V"))
        n = case["B"] * case.get("T", 1)
        qk, v, h = n * Hq * K * e, n * Hv * V * e, n * Hv * e
        if op.endswith("step"):
            live = case["B"] - case["pad"]
            return {"bytes": 2 * qk + 2 * v + 2 * h + 8 * live * Hv * K * V, "flops": (8 if op == "delta_step" else 6) * live * Hv * K * V}
        st = (case["N"] or case["B"]) * Hv * K * V * 4
        # products of the chunked form: C B^T (once a group), P x, C S, B^T x; backward twice those and the state again
        f = n * (2 * CHUNK * Hq * K + Hv * (2 * CHUNK * V + 4 * K * V))
        if op == "scan_fwd":
            return {"bytes": 2 * qk + 2 * v + h + st * (1 + case["state"]), "flops": f}
        return {"bytes": 4 * qk + 3 * v + 2 * h + 3 * st * case["state"], "flops": 2 * f + n * Hv * (2 * CHUNK * V + 4 * K * V)}
    n, r = case["rows"] * case["D"], case["rows"] * 4 * (2 - case["rms"])
    if op == "norm_fwd":
        return {"bytes": n * e * (2 + case["gate"]) + r, "flops": 8 * n}
    return {"bytes": n * e * (3 + 2 * case["gate"]) + r, "flops": 16 * n}


# ---------------------------------------------------------------- in 64 bits, from the definitions


def _spans(s):
    """(row of the state, first token, end) of every sequence, tokens counted over all rows."""
    case = s["case"]
    if s["cu"] is not None:
        return [(n, p, q) for n, (p, q) in enumerate(zip(s["cuts"], s["cuts"][1:]))]
    return [(n, n * case["T"], (n + 1) * case["T"]) for n in range(case["B"])]


def _d(t):
    return None if t is None else t.double()


def _conv_exact(s):
    case, W = s["case"], s["case"]["W"]
    D = case["D"]
    x, w = s["x"].double().reshape(-1, D), s["weight"].double()
    bias = 0 if s["bias"] is None else s["bias"].double()
    back = case["op"] == "conv_bwd"
    out, ht = torch.zeros_like(x), x.new_zeros(case["N"] or case["B"], W - 1, D)
    dx, dw, db, dh = torch.zeros_like(x), torch.zeros_like(w), x.new_zeros(D), torch.zeros_like(ht)
    for n, p, q in _spans(s):
        old = x.new_zeros(W - 1, D) if s["h0"] is None else s["h0"][n].double()
        z = torch.cat([old, x[p:q]])
        L = q - p
        pre = bias + sum(z[j:j + L] * w[:, j] for j in range(W))
        sg = 1 / (1 + torch.exp(-pre))
        if not back:
            out[p:q] = pre * sg if case["silu"] else pre
            ht[n] = z[L:]
            continue
        d = s["dy"].double().reshape(-1, D)[p:q]
        d = d * sg * (1 + pre * (1 - sg)) if case["silu"] else d
        dz = torch.zeros_like(z)
        if s["dht"] is not None:
            dz[L:] += s["dht"][n].double()
        for j in range(W):
            dz[j:j + L] += d * w[:, j]
            dw[:, j] += (d * z[j:j + L]).sum(0)
        db += d.sum(0)
        dx[p:q], dh[n] = dz[W - 1:], dz[:W - 1]
    if not back:
        return out.reshape(s["x"].shape), ht
    return [dx.reshape(s["x"].shape), dw, None if s["bias"] is None else db, None if s["h0"] is None else dh]


def _scan_exact(s):
    """Each head by itself as one lower triangular matrix over a sequence's tokens."""
    case = s["case"]
    Hq, Hv, K, V = (case[k] for k in ("Hq", "Hv", "K", "V"))
    c, b = (s[k].double().reshape(-1, Hq, K) for k in ("c", "b"))
    x = s["x"].double().reshape(-1, Hv, V)
    z = s["dt"].double().reshape(-1, Hv) + (0 if s["dt_bias"] is None else s["dt_bias"].double())
    delta = torch.logaddexp(z, torch.zeros_like(z)) if case["softplus"] else z
    back = case["op"] == "scan_bwd"
    rows = case["N"] or case["B"]
    y, ht = torch.zeros_like(x), x.new_zeros(rows, Hv, K, V)
    dy = s["dy"].double().reshape(-1, Hv, V) if back else None
    dc, db, dx, ddel = torch.zeros_like(c), torch.zeros_like(b), torch.zeros_like(x), torch.zeros_like(z)
    dA, dD, dh = x.new_zeros(Hv), x.new_zeros(Hv), torch.zeros_like(ht)
    for n, p, q in _spans(s):
        for h in range(Hv):
            u = h // (Hv // Hq)
            a, D = s["A"][h].double(), 0 if s["D"] is None else s["D"][h].double()
            h0 = x.new_zeros(K, V) if s["h0"] is None else s["h0"][n, h].double()
            R = s["dht"][n, h].double() if back and s["dht"] is not None else x.new_zeros(K, V)
            if p == q:
                ht[n, h], dh[n, h] = h0, R
                continue
            de = delta[p:q, h]
            gam = torch.cumsum(de * a, 0)
            ci, bi, xi = c[p:q, u], b[p:q, u], x[p:q, h]
            E = (gam[:, None] - gam[None, :]).tril_()
            E = E.exp_().tril_()
            G = ci @ bi.T
            start, end = torch.exp(gam)[:, None], torch.exp(gam[-1] - gam)
            if not back:
                y[p:q, h] = (E * G * de) @ xi + start * (ci @ h0) + D * xi
                ht[n, h] = start[-1] * h0 + (bi * (end * de)[:, None]).T @ xi
                continue
            d = dy[p:q, h]
            M = d @ xi.T
            EG = E * G
            dx[p:q, h] = de[:, None] * (EG.T @ d + end[:, None] * (bi @ R)) + D * d
            EG *= M
            E *= M
            E *= de
            tail = end * ((bi @ R) * xi).sum(-1)  # of the token's part in the final state
            head = start[:, 0] * ((ci @ h0) * d).sum(-1)
            dc[p:q, u] += E @ bi + start * (d @ h0.T)
            db[p:q, u] += E.T @ ci + (end * de)[:, None] * (xi @ R.T)
            direct = EG.sum(0) + tail
            final = start[-1] * h0 + (bi * (end * de)[:, None]).T @ xi
            dgam = (EG * de).sum(1) + head - de * direct
            dgam[-1] += (R * final).sum()
            dg = torch.flip(torch.cumsum(torch.flip(dgam, [0]), 0), [0])
            ddel[p:q, h] = direct + a * dg
            dA[h] += (de * dg).sum()
            dD[h] += (d * xi).sum()
            dh[n, h] = (ci * start).T @ d + start[-1] * R
    if not back:
        return y.reshape(s["x"].shape), ht
    ddt = ddel / (1 + torch.exp(-z)) if case["softplus"] else ddel
    like = [dc.reshape(s["c"].shape), db.reshape(s["b"].shape), dx.reshape(s["x"].shape), ddt.reshape(s["dt"].shape)]
    return like + [dA, None if s["D"] is None else dD, None if s["dt_bias"] is None else ddt.sum(0), None if s["h0"] is None else dh]


def _step_exact(s):
    case, op = s["case"], s["case"]["op"]
    B, live = case["B"], case["B"] - case["pad"]
    at = list(range(B)) if s["index"] is None else s["index"].tolist()
    S = s["state"].double()
    old = S[at[:live]]
    if op == "conv_step":
        W = case["W"]
        x, w = s["x"].double(), s["weight"].double()
        pre = x[:live] * w[:, W - 1] + sum(old[:, j] * w[:, j] for j in range(W - 1))
        pre = pre if s["bias"] is None else pre + s["bias"].double()
        y = torch.zeros_like(x)
        y[:live] = pre / (1 + torch.exp(-pre)) if case["silu"] else pre
        S[at[:live]] = torch.cat([old[:, 1:], x[:live, None]], 1)
        return y, S
    of = torch.arange(case["Hv"], device=S.device) // (case["Hv"] // case["Hq"])
    if op == "scan_step":
        c, b, x = s["c"].double()[:live, of], s["b"].double()[:live, of], s["x"].double()
        z = s["dt"].double()[:live] + (0 if s["dt_bias"] is None else s["dt_bias"].double())
        de = torch.logaddexp(z, torch.zeros_like(z)) if case["softplus"] else z
        new = old * torch.exp(de * s["A"].double())[:, :, None, None] + de[:, :, None, None] * b[:, :, :, None] * x[:live, :, None, :]
        y = torch.zeros_like(x)
        y[:live] = torch.matmul(c[:, :, None, :], new)[:, :, 0] + (0 if s["D"] is None else s["D"].double()[:, None] * x[:live])
    else:
        q, k = s["q"].double()[:live, of], s["k"].double()[:live, of]
        if case["l2norm"]:
            q, k = (t / torch.sqrt((t ** 2).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        v, be = s["v"].double(), s["beta"].double()[:live, :, None]
        old = old * torch.exp(s["g"].double()[:live])[:, :, None, None]
        new = old + k[..., :, None] * (be * (v[:live] - torch.matmul(k[:, :, None, :], old)[:, :, 0]))[..., None, :]
        y = torch.zeros_like(v)
        y[:live] = torch.matmul(q[:, :, None, :], new)[:, :, 0] / case["K"] ** 0.5
    S[at[:live]] = new
    return y, S


def _norm_exact(s):
    case = s["case"]
    x, gate = s["x"].double(), _d(s["gate"])
    one = x.new_ones(case["D"]) if s["weight"] is None else s["weight"].double()
    off = 0 if s["bias"] is None else s["bias"].double()
    mean = x.new_zeros(x.shape[0]) if case["rms"] else x.mean(1)
    mid = x - mean[:, None]
    rstd = 1 / torch.sqrt((mid * mid).mean(1) + EPS)
    hat = mid * rstd[:, None]
    z = hat * one + off
    sg = None if gate is None else 1 / (1 + torch.exp(-gate))
    if case["op"] == "norm_fwd":
        return z if gate is None else z * gate * sg, None if case["rms"] else mean, rstd
    dy = s["dy"].double()
    dz = dy if gate is None else dy * gate * sg
    dgate = None if gate is None else dy * z * sg * (1 + gate * (1 - sg))
    t = dz * one
    dx = t - hat * (t * hat).mean(1, keepdim=True)
    if not case["rms"]:
        dx = dx - t.mean(1, keepdim=True)
    return [dx * rstd[:, None], None if s["weight"] is None else (dz * hat).sum(0), None if s["bias"] is None else dz.sum(0), dgate]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv_fwd", "conv_bwd"):
        return _conv_exact(s)
    if op in ("scan_fwd", "scan_bwd"):
        return _scan_exact(s)
    return _step_exact(s) if op.endswith("_step") else _norm_exact(s)
