"""What linear attention with a decay for each head and the group norm are measured on.

Operators: linear attention with one decay a head (prompt, backward, single token), and group norm over
channels-last tensors with an activation or an output gate (forward, backward).  With ``own`` false ``run``
computes them from elementary torch operations in 32 bits; with ``own`` true it makes the library's calls.

A case is a dict of plain values:
  op      attn_fwd | attn_bwd | attn_step | group_fwd | group_bwd
  dtype   bf16 | f32
  B, T    batch rows and tokens each; with N > 0 one packed batch of T tokens cut into N sequences at
          places that ``cut`` (a seed) gives, some of them empty or one token long
  N, S    group norm: samples and positions of each; statistics are over the S positions and the channels of a group
  others  sizes and switches of the operator
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64
EPS = 1e-5


def listed():
    return [
        # a long prompt through one layer, 64 heads of 128
        {"name": "attn_prompt_bf16", "op": "attn_fwd", "dtype": "bf16", "B": 1, "T": 8192, "N": 0, "cut": 0, "Hq": 64, "Hv": 64,
         "K": 128, "V": 128, "state": False},
        # prompts of a serving batch, packed, that go on from saved states; two v-heads share a q and a k head
        {"name": "attn_prompts_bf16", "op": "attn_fwd", "dtype": "bf16", "B": 1, "T": 16384, "N": 16, "cut": 170, "Hq": 16, "Hv": 32,
         "K": 128, "V": 128, "state": True},
        # a few short prompts of odd lengths in full precision
        {"name": "attn_prompts_f32", "op": "attn_fwd", "dtype": "f32", "B": 1, "T": 1277, "N": 7, "cut": 3, "Hq": 2, "Hv": 8,
         "K": 64, "V": 64, "state": True},
        # one training step's backward over two rows of 4096, 32 heads of 128
        {"name": "attn_train_bf16", "op": "attn_bwd", "dtype": "bf16", "B": 2, "T": 4096, "N": 0, "cut": 0, "Hq": 32, "Hv": 32,
         "K": 128, "V": 128, "state": False},
        # a backward over packed sequences of odd lengths with states, heads of 64 in pairs, in full precision
        {"name": "attn_train_f32", "op": "attn_bwd", "dtype": "f32", "B": 1, "T": 1901, "N": 5, "cut": 2, "Hq": 4, "Hv": 8,
         "K": 64, "V": 64, "state": True},
        # one generated token of one request: latency
        {"name": "attn_token_one_bf16", "op": "attn_step", "dtype": "bf16", "B": 1, "Hq": 32, "Hv": 32, "K": 128, "V": 128,
         "pool": 0, "pad": 0},
        # a full decode batch whose states lie in a pool of slots
        {"name": "attn_token_pool_bf16", "op": "attn_step", "dtype": "bf16", "B": 250, "Hq": 32, "Hv": 32, "K": 128, "V": 128,
         "pool": 256, "pad": 5},
        # the gated norm of each head of the attention's output, token by token: 8192 tokens, 64 heads of 128
        {"name": "group_heads_bf16", "op": "group_fwd", "dtype": "bf16", "N": 8192, "S": 1, "G": 64, "Dg": 128, "gate": True,
         "silu": False, "affine": True},
        # the same norm's backward in a training step
        {"name": "group_heads_train_bf16", "op": "group_bwd", "dtype": "bf16", "N": 8192, "S": 1, "G": 64, "Dg": 128, "gate": True,
         "silu": False, "affine": True},
        # a norm with SiLU over whole maps of 96 x 96 positions, 320 channels in 32 groups
        {"name": "group_maps_bf16", "op": "group_fwd", "dtype": "bf16", "N": 8, "S": 9216, "G": 32, "Dg": 10, "gate": False,
         "silu": True, "affine": True},
        # the backward over maps of 64 x 64 positions, 512 channels in 32 groups
        {"name": "group_maps_train_bf16", "op": "group_bwd", "dtype": "bf16", "N": 6, "S": 4096, "G": 32, "Dg": 16, "gate": False,
         "silu": True, "affine": True},
        # a small map of odd sizes in full precision, backward
        {"name": "group_train_f32", "op": "group_bwd", "dtype": "f32", "N": 3, "S": 333, "G": 11, "Dg": 7, "gate": False,
         "silu": True, "affine": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step", "group_fwd", "group_fwd", "group_bwd", "group_bwd"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    packed = rng.random() < 0.5
    if op in ("attn_fwd", "attn_bwd"):
        Hq = rng.choice([1, 2, 3, 4, 8, 16])
        Hv = Hq * rng.choice([1, 1, 2, 3, 4])
        T = _log(rng, 1, min(16384, (1 << 18) // Hv, 2048 if c["dtype"] == "f32" else 16384))
        c |= {"B": 1 if packed else rng.choice([1, 2, 3]), "N": _log(rng, 1, 16) if packed else 0, "cut": rng.randrange(1 << 20),
              "Hq": Hq, "Hv": Hv, "K": rng.choice([32, 64, 128]), "V": rng.choice([32, 64, 128]), "state": rng.random() < 0.5}
        c["T"] = T if packed else max(1, T // c["B"])
    elif op == "attn_step":
        Hq = _log(rng, 1, 16)
        c |= {"B": _log(rng, 1, 150), "Hq": Hq, "Hv": Hq * rng.choice([1, 2, 3]), "K": rng.choice([32, 64, 128]),
              "V": rng.choice([32, 64, 128])}
        c |= {"pool": c["B"] + rng.randrange(1, 9), "pad": rng.randrange(0, (c["B"] + 1) // 2)} if packed else {"pool": 0, "pad": 0}
    else:
        G, Dg = _log(rng, 1, 64), _log(rng, 1, 160)
        S = 1 if rng.random() < 0.3 else _log(rng, 2, min(16384, (1 << 25) // (G * Dg)))
        Dg = max(Dg if rng.random() < 0.5 else (Dg + 7) // 8 * 8, 16 // S)  # (two values normalised leave only their sign)
        gate = rng.random() < 0.4
        c |= {"N": _log(rng, 1, min(16384, max(1, (1 << 25) // (G * Dg * S)))), "S": S, "G": G, "Dg": Dg,
              "gate": gate, "silu": not gate and rng.random() < 0.7, "affine": rng.random() < 0.8}
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

    def act(*shape):  # q and k come through a SiLU
        z = torch.randn(*shape, generator=gen, device="cuda")
        return (z * torch.sigmoid(z)).to(dt)

    f32 = torch.float32
    s = {"case": case, "cu": None}
    if op.startswith("attn"):
        Hq, Hv, K, V = (case[k] for k in ("Hq", "Hv", "K", "V"))
        step = op == "attn_step"
        if not step and case["N"]:
            s["cuts"] = _cuts(case)
            s["cu"] = torch.tensor(s["cuts"], dtype=torch.int32, device="cuda")
        lead = (case["B"],) if step else (case["B"], case["T"])
        s["q"], s["k"], s["v"] = act(*lead, Hq, K), act(*lead, Hq, K), normal(*lead, Hv, V)
        # slopes from 2^-(8 / Hv) to 2^-8 a token, less for the later of a model's layers: `layer` is this layer's share
        layer = 0.1 + 0.9 * torch.rand(1, generator=gen, device="cuda")
        s["log_decay"] = -layer * torch.exp2(-8 * (torch.arange(Hv, device="cuda", dtype=f32) + 1) / Hv)
        if step:
            slots = case["pool"] or case["B"]
            s["index"] = None
            if case["pool"]:
                s["index"] = torch.randperm(slots, generator=gen, device="cuda")[: case["B"]].to(torch.int32)
                s["index"][case["B"] - case["pad"]:] = -1
            s["state"] = normal(slots, Hv, K, V, like=f32)
            return s
        rows = case["N"] or case["B"]
        s["h0"] = normal(rows, Hv, K, V, like=f32) if case["state"] else None
        if op == "attn_bwd":
            s["do"] = normal(*lead, Hv, V)
            s["dht"] = 0.1 * normal(rows, Hv, K, V, like=f32) if case["state"] else None
        return s
    N, S, C = case["N"], case["S"], case["G"] * case["Dg"]
    shape = (N, C) if S == 1 else (N, S, C)
    lead = (N,) + (1,) * (len(shape) - 1)
    s["x"] = (normal(*shape, like=f32) * torch.exp(0.5 * normal(*lead, like=f32)) + 0.3).to(dt)
    s["weight"] = 1 + 0.1 * normal(C, like=f32) if case["affine"] else None
    s["bias"] = 0.1 * normal(C, like=f32) if case["affine"] else None
    s["gate"] = normal(*shape) if case["gate"] else None
    if op == "group_bwd":  # what the forward left
        s["dy"] = normal(*shape)
        x = s["x"].double().reshape(N, S, case["G"], case["Dg"])
        s["mean"] = x.mean((1, 3)).float()
        s["rstd"] = ((x - x.mean((1, 3), keepdim=True)) ** 2).mean((1, 3)).add(EPS).rsqrt().float()
    return s


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


def _attn(s, q, k, v, h0):
    """Chunks of 64 tokens: products inside a chunk, and the states between chunks from the tokens between them."""
    case, g = s["case"], s["log_decay"].double()
    (B, T), (Hq, Hv, K, V) = v.shape[:2], (case[n] for n in ("Hq", "Hv", "K", "V"))
    rows, dev = case["N"] or B, v.device
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(B + 1, device=dev) * T
    L = max([b - a for a, b in zip(s["cuts"], s["cuts"][1:])]) if s["cu"] is not None else T
    nc = (L + CHUNK - 1) // CHUNK
    at = cu[:-1, None] + torch.arange(nc * CHUNK, device=dev)  # every sequence padded to nc chunks
    live = at < cu[1:, None]
    at = torch.clamp(at, max=B * T - 1)

    def cut(t):  # [B, T, H, ..] -> [rows, nc, H, CHUNK, ..], zeros behind a sequence's end
        t = t.reshape(B * T, *t.shape[2:])[at] * live[..., None, None]
        return t.reshape(rows, nc, CHUNK, *t.shape[2:]).transpose(2, 3)

    i = torch.arange(CHUNK, device=dev)
    far = (i[:, None] - i[None, :]).double()
    R = Hv // Hq
    q, k, v = cut(q * K ** -0.5), cut(k), cut(v)
    E = torch.exp(torch.where(far < 0, float("-inf"), far * g[:, None, None])).float()
    P = (q @ k.transpose(-1, -2)).repeat_interleave(R, 2) * E
    before = torch.minimum(torch.arange(nc + 1, device=dev) * CHUNK, (cu[1:] - cu[:-1])[:, None])  # tokens before each chunk
    left = torch.clamp(before[:, 1:, None] - before[:, :-1, None] - 1 - i, min=0)  # tokens behind a token in its chunk
    w = torch.exp(left[:, :, None].double() * g[:, None]).float()
    U = (k.transpose(-1, -2).repeat_interleave(R, 2) * w[..., None, :]) @ v  # what each chunk adds to the state
    ends = torch.cat([before.new_zeros(rows, 1), before[:, 1:]], 1)  # tokens before the end of each of a state's terms
    gap = before[:, :, None] - ends[:, None, :]
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=dev).tril()
    W = torch.exp(torch.where(low, gap.double()[:, None] * g[:, None, None], float("-inf"))).float()  # [rows, Hv, nc + 1, nc + 1]
    h0 = v.new_zeros(rows, Hv, K, V) if h0 is None else h0
    S = (W @ torch.cat([h0[:, None], U], 1).transpose(1, 2).reshape(rows, Hv, nc + 1, K * V)).reshape(rows, Hv, nc + 1, K, V)
    start = torch.exp((i + 1).double() * g[:, None]).float()
    o = P @ v + start[..., None] * (q.repeat_interleave(R, 2) @ S[:, :, :nc].transpose(1, 2).contiguous())
    o = o.transpose(2, 3).reshape(rows, nc * CHUNK, Hv, V)
    t = torch.arange(B * T, device=dev)
    n = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[n, t - cu[n]].reshape(B, T, Hv, V), S[:, :, nc]


def _group(s, x, weight, bias, gate):
    case = s["case"]
    N, S, G, Dg = (case[k] for k in ("N", "S", "G", "Dg"))
    z = x.reshape(N, S, G, Dg)
    mean = z.mean((1, 3), keepdim=True)
    rstd = torch.rsqrt(((z - mean) ** 2).mean((1, 3), keepdim=True) + EPS)
    y = ((z - mean) * rstd).reshape(x.shape)
    y = y if weight is None else y * weight + bias
    y = _silu(y) if case["silu"] else y
    return y if gate is None else y * _silu(gate), mean.reshape(N, G), rstd.reshape(N, G)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DT[case["dtype"]]
    if op == "attn_fwd":
        o, ht = _attn(s, *(_f(s[k]) for k in ("q", "k", "v", "h0")))
        return o.to(dt), ht
    if op == "attn_bwd":
        return _grad(lambda *a: _attn(s, *a), [s[k] for k in ("q", "k", "v", "h0")], [s["do"], s["dht"]])
    if op == "attn_step":
        live, R = case["B"] - case["pad"], case["Hv"] // case["Hq"]
        at = slice(0, live) if s["index"] is None else s["index"][:live].long()
        q, k, v = (s[n][:live].float() for n in ("q", "k", "v"))
        S = torch.exp(s["log_decay"])[:, None, None] * s["state"][at] + k.repeat_interleave(R, 1)[..., :, None] * v[..., None, :]
        o = case["K"] ** -0.5 * (S * q.repeat_interleave(R, 1)[..., :, None]).sum(-2)
        s["state"][at] = S
        return torch.cat([o, o.new_zeros(case["pad"], *o.shape[1:])]).to(dt), s["state"]
    args = [s[k] for k in ("x", "weight", "bias", "gate")]
    if op == "group_fwd":
        y, mean, rstd = _group(s, *map(_f, args))
        return y.to(dt), mean, rstd
    return _grad(lambda *a: _group(s, *a), args, [s["dy"], None, None])


# ---------------------------------------------------------------- the library's calls


def _library(s):
    import gated_deltanet_chunked_gdn_amd as gdn
    case, op = s["case"], s["case"]["op"]
    if op == "attn_fwd":
        return gdn.linear_attention_fwd(s["q"], s["k"], s["v"], s["log_decay"], initial_state=s["h0"], cu_seqlens=s["cu"],
                                        check_cu_seqlens=False)
    if op == "attn_bwd":
        return gdn.linear_attention_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], dht=s["dht"], initial_state=s["h0"],
                                        cu_seqlens=s["cu"], check_cu_seqlens=False)
    if op == "attn_step":
        return gdn.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], state_indices=s["index"]), s["state"]
    act = "silu" if case["silu"] else None
    if op == "group_fwd":
        return gdn.group_norm_fwd(s["x"], case["G"], s["weight"], s["bias"], gate=s["gate"], activation=act, eps=EPS)
    return gdn.group_norm_bwd(s["dy"], s["x"], case["G"], s["weight"], s["bias"], s["mean"], s["rstd"], gate=s["gate"], activation=act)


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- sizes


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("attn"):
        Hq, Hv, K, V = (case[k] for k in ("Hq", "Hv", "K", "V"))
        n = case["B"] * case.get("T", 1)
        qk, v = n * Hq * K * e, n * Hv * V * e
        if op == "attn_step":
            live = case["B"] - case["pad"]
            return {"bytes": 2 * qk + 2 * v + 8 * live * Hv * K * V, "flops": 6 * live * Hv * K * V}
        st = (case["N"] or case["B"]) * Hv * K * V * 4
        # products of the chunked form: Q K^T (once a group), P V, Q S, K^T V; backward three like these
        f = n * (2 * CHUNK * Hq * K + Hv * (2 * CHUNK * V + 4 * K * V))
        if op == "attn_fwd":
            return {"bytes": 2 * qk + 2 * v + st * (1 + case["state"]), "flops": f}
        return {"bytes": 4 * qk + 3 * v + 3 * st * case["state"], "flops": 3 * f}
    n, r = case["N"] * case["S"] * case["G"] * case["Dg"], case["N"] * case["G"] * 8
    if op == "group_fwd":
        return {"bytes": n * e * (2 + case["gate"]) + r, "flops": 8 * n}
    return {"bytes": n * e * (3 + 2 * case["gate"]) + r, "flops": 16 * n}


# ---------------------------------------------------------------- in 64 bits, from the definitions


def _attn_exact(s):
    """Each head by itself as one lower triangular matrix over a sequence's tokens."""
    case = s["case"]
    Hq, Hv, K, V = (case[k] for k in ("Hq", "Hv", "K", "V"))
    q, k = (s[n].double().reshape(-1, Hq, K) for n in ("q", "k"))
    v = s["v"].double().reshape(-1, Hv, V)
    back = case["op"] == "attn_bwd"
    rows = case["N"] or case["B"]
    borders = s["cuts"] if s["cu"] is not None else [n * case["T"] for n in range(case["B"] + 1)]
    o, ht = torch.zeros_like(v), v.new_zeros(rows, Hv, K, V)
    dq, dk, dv, dh = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(ht)
    do = s["do"].double().reshape(-1, Hv, V) if back else None
    for n, (a, b) in enumerate(zip(borders, borders[1:])):
        t = torch.arange(b - a, device=v.device, dtype=torch.float64)
        far = t[:, None] - t[None, :]
        for h in range(Hv):
            u, g = h // (Hv // Hq), s["log_decay"][h].double()
            h0 = v.new_zeros(K, V) if s["h0"] is None else s["h0"][n, h].double()
            R = s["dht"][n, h].double() if back and s["dht"] is not None else v.new_zeros(K, V)
            qi, ki, vi = q[a:b, u] / K ** 0.5, k[a:b, u], v[a:b, h]
            M = (far * g).exp_().tril_()
            first, last, whole = torch.exp((t + 1) * g)[:, None], torch.exp((b - a - 1 - t) * g)[:, None], torch.exp((b - a) * g)
            if not back:
                M *= qi @ ki.T
                o[a:b, h] = M @ vi + first * (qi @ h0)
                ht[n, h] = whole * h0 + (last * ki).T @ vi
                continue
            d = do[a:b, h]
            dv[a:b, h] = (M * (qi @ ki.T)).T @ d + last * (ki @ R)
            M *= d @ vi.T
            dq[a:b, u] += (M @ ki + first * (d @ h0.T)) / K ** 0.5
            dk[a:b, u] += M.T @ qi + last * (vi @ R.T)
            dh[n, h] = whole * R + (first * qi).T @ d
    if not back:
        return o.reshape(s["v"].shape), ht
    return [dq.reshape(s["q"].shape), dk.reshape(s["k"].shape), dv.reshape(s["v"].shape), None if s["h0"] is None else dh]


def _step_exact(s):
    case = s["case"]
    live = case["B"] - case["pad"]
    at = list(range(live)) if s["index"] is None else s["index"].tolist()[:live]
    of = torch.arange(case["Hv"], device="cuda") // (case["Hv"] // case["Hq"])
    q, k, v = s["q"].double()[:live, of], s["k"].double()[:live, of], s["v"].double()
    S = s["state"].double()
    new = S[at] * torch.exp(s["log_decay"].double())[None, :, None, None] + k[..., :, None] * v[:live, :, None, :]
    o = torch.zeros_like(v)
    o[:live] = torch.matmul(q[:, :, None, :], new)[:, :, 0] / case["K"] ** 0.5
    S[at] = new
    return o, S


def _group_exact(s):
    case = s["case"]
    N, S, G, Dg = (case[k] for k in ("N", "S", "G", "Dg"))
    x = s["x"].double().reshape(N, S, G, Dg)
    w = x.new_ones(G, Dg) if s["weight"] is None else s["weight"].double().reshape(G, Dg)
    off = x.new_zeros(G, Dg) if s["bias"] is None else s["bias"].double().reshape(G, Dg)
    gate = None if s["gate"] is None else s["gate"].double().reshape(x.shape)
    count = S * Dg
    mean = x.sum((1, 3)) / count
    mid = x - mean[:, None, :, None]
    rstd = 1 / torch.sqrt((mid * mid).sum((1, 3)) / count + EPS)
    hat = mid * rstd[:, None, :, None]
    z = hat * w + off
    sz = 1 / (1 + torch.exp(-z))
    sg = None if gate is None else 1 / (1 + torch.exp(-gate))
    y = z * sz if case["silu"] else z
    if case["op"] == "group_fwd":
        y = y if gate is None else y * gate * sg
        return y.reshape(s["x"].shape), mean, rstd
    dy = s["dy"].double().reshape(x.shape)
    dgate = None if gate is None else dy * y * sg * (1 + gate * (1 - sg))
    dz = dy if gate is None else dy * gate * sg
    dz = dz * sz * (1 + z * (1 - sz)) if case["silu"] else dz
    t = dz * w
    dx = t - t.sum((1, 3), keepdim=True) / count - hat * (t * hat).sum((1, 3), keepdim=True) / count
    dx = (dx * rstd[:, None, :, None]).reshape(s["x"].shape)
    none = s["weight"] is None
    return [dx, None if none else (dz * hat).sum((0, 1)).reshape(-1), None if none else dz.sum((0, 1)).reshape(-1),
            None if dgate is None else dgate.reshape(s["x"].shape)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn_step":
        return _step_exact(s)
    return _attn_exact(s) if case["op"].startswith("attn") else _group_exact(s)
