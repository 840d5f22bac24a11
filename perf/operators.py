"""Linear attention with a decay for each head, and rotary positions: the cases that are measured, in plain torch
operations (``own`` false) and through the library (``own`` true).

Per batch row and head, with lam = exp(log_decay[h]) and float32 states of D x M:

    S_t = lam S_{t-1} + k_t v_t^T,    out_t = scale * q_t^T S_t

Four kinds of case:

* ``prompt``: a whole sequence at once, from a state or the empty one, to the outputs and the state after it;
* ``train``: the same, then the gradients of q, k and v (and of the state) for a given gradient of the outputs;
* ``step``: one token for each of N sequences against their states;
* ``rotary``: the rotation of q and k by their positions, or its gradient (the inverse rotation).
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ---

def _attention(name, kind, B, T, H, D, M, dtype, lengths=False, state=False):
    return {"name": name, "kind": kind, "B": B, "T": T, "H": H, "D": D, "M": M, "dtype": dtype,
            "lengths": lengths, "state": state}


def _rotary(name, B, T, Hq, Hk, D, R, dtype, interleaved, scaling, inverse, far):
    return {"name": name, "kind": "rotary", "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "dtype": dtype,
            "interleaved": interleaved, "scaling": scaling, "inverse": inverse, "far": far}


def listed():
    return [
        # a chat prompt of one user on a 768-wide layer: everything is latency
        _attention("prompt_short", "prompt", 1, 199, 12, 64, 64, "bf16"),
        # eight prompts of different lengths, padded into one batch, on a 2048-wide layer; each continues a state
        _attention("prompt_ragged", "prompt", 8, 4096, 16, 128, 128, "bf16", lengths=True, state=True),
        # one book-long prompt on a 2560-wide layer: few heads, many positions
        _attention("prompt_long", "prompt", 1, 65536, 20, 128, 128, "bf16"),
        # a 768-wide layer evaluated in float32
        _attention("prompt_f32", "prompt", 8, 1024, 12, 64, 64, "f32", state=True),
        # a training step's attention on a 768-wide layer
        _attention("train_768", "train", 8, 1024, 12, 64, 64, "bf16"),
        # the same on a 2048-wide layer with long sequences
        _attention("train_2048", "train", 8, 4096, 16, 128, 128, "bf16"),
        # float32 training on sequences of an odd length that continue a state (gradients reach the state)
        _attention("train_f32", "train", 2, 1001, 12, 64, 64, "f32", state=True),
        # one user's next token on a 768-wide layer
        _attention("step_one", "step", 1, 1, 12, 64, 64, "bf16"),
        # 512 users' next tokens on a 5120-wide layer: the states' traffic
        _attention("step_many", "step", 512, 1, 40, 128, 128, "bf16"),
        # positions of one decode step for 512 users, far into their texts, frequencies scaled by parts
        _rotary("rotary_step", 512, 1, 40, 40, 128, 128, "bf16", False, "by_parts", False, 1 << 20),
        # queries and keys of a training batch on a 2048-wide layer, half of each head rotated
        _rotary("rotary_batch", 8, 4096, 16, 16, 128, 64, "bf16", False, "none", False, 0),
        # the gradient of the interleaved form in float32 on a 768-wide layer
        _rotary("rotary_grad", 8, 1024, 12, 12, 64, 64, "f32", True, "linear", True, 1 << 15),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    kind = rng.choice(["prompt", "train", "step", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "rotary":
        D = rng.choice([32, 64, 80, 96, 128])
        B, T = _log_int(rng, 1, 512), _log_int(rng, 1, 16384)
        H = rng.choice([1, 3, 8, 12, 16, 40])
        Hk = rng.choice([1, H])
        while B * T * (H + Hk) * D > 8 * 4096 * 32 * 128:
            B, T = (B + 1) // 2, (3 * T + 3) // 4
        R = rng.choice([D, D // 2, D - 16])
        return _rotary("", B, T, H, Hk, D, R, dtype, rng.random() < 0.5,
                       rng.choice(["none", "linear", "ntk", "by_parts"]), rng.random() < 0.3,
                       rng.choice([0, 1 << 12, 1 << 20]))
    D, M = rng.choice([32, 64, 72, 96, 128]), rng.choice([32, 64, 72, 96, 128])
    H = rng.choice([1, 4, 8, 12, 16, 20, 40])
    if kind == "step":
        N = _log_int(rng, 1, 512)
        return _attention("", "step", N, 1, H, D, M, dtype)
    B, T = _log_int(rng, 1, 64), _log_int(rng, 1, 65536 if kind == "prompt" else 8192)
    most = 8 * 4096 * 16 * 128 * 128
    while B * T * H * D * M > most // (1 if dtype == "bf16" else 4):
        B, T = (B + 1) // 2, (3 * T + 3) // 4
    return _attention("", kind, B, T, H, D, M, dtype, lengths=rng.random() < 0.4, state=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs ---

def _frequencies(R, scaling):
    """Angular frequencies per position (float64) and the factor on the rotated pair: base 10000; by a factor of 8:
    positions compressed (linear), the base raised (ntk), or compressed only where a pair turns slowly (by_parts)."""
    i = torch.arange(0, R, 2, dtype=torch.float64)
    factor = 8.0
    base = 10000.0 * (factor ** (R / (R - 2)) if scaling == "ntk" and R > 2 else 1.0)
    f = base ** (-i / R)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    return f, mscale


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device=dev, dtype=torch.float32, generator=gen)

    s = {"case": case}
    B, T = case["B"], case["T"]
    if case["kind"] == "rotary":
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        # queries, keys and values lie side by side, as one projection leaves them
        qkv = normal(B, T, (Hq + 2 * Hk) * D).to(dt)
        s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = qkv[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        first = torch.randint(0, case["far"] + 1, (B, 1), device=dev, generator=gen)
        s["positions"] = first + torch.arange(T, device=dev)
        f, s["mscale"] = _frequencies(case["R"], case["scaling"])
        s["inv_freq"] = f.to(dev)
        return s
    H, D, M = case["H"], case["D"], case["M"]
    qkv = normal(B, T, H * (2 * D + M)).to(dt)
    s["q"] = qkv[..., :H * D].unflatten(-1, (H, D))
    s["k"] = qkv[..., H * D:2 * H * D].unflatten(-1, (H, D))
    s["v"] = qkv[..., 2 * H * D:].unflatten(-1, (H, M))
    # memories of one or two positions to several hundred, spread over the heads
    h = torch.arange(1, H + 1, device=dev, dtype=torch.float32)
    s["log_decay"] = -torch.exp2(-8.0 * h / H) * (0.5 + torch.rand(H, device=dev, generator=gen))
    s["scale"] = D ** -0.5
    if case["kind"] == "step":
        s["q"], s["k"], s["v"] = s["q"][:, 0], s["k"][:, 0], s["v"][:, 0]
        s["state"] = normal(B, H, D, M)
        s["state_out"] = torch.empty_like(s["state"])
        return s
    s["state"] = normal(B, H, D, M) if case["state"] else None
    s["lengths"] = None
    if case["lengths"]:
        s["lengths"] = torch.randint(T // 4, T + 1, (B,), device=dev, generator=gen, dtype=torch.int32)
    if case["kind"] == "train":
        s["grad_out"] = normal(B, T, H, M).to(dt)
        s["grad_state"] = normal(B, H, D, M) if case["state"] else None
    return s


# ------------------------------------------------------------- plain form ---

_CHUNK = 128


def _plain_scan(a, b, c, g, state, scale):
    """out_t = scale * (sum_{j<=t} lam^{t-j} (a_t . b_j) c_j + lam^{t+1} a_t^T state) for float32 a, b [B, H, T, X] and
    c [B, H, T, Y], in chunks: products inside a chunk, and the states at the chunks' starts from one product over
    chunks."""
    B, H, T, X = a.shape
    Y = c.shape[-1]
    n = (T + _CHUNK - 1) // _CHUNK
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, n * _CHUNK - T)).unflatten(2, (n, _CHUNK)) for x in (a, b, c))
    i = torch.arange(_CHUNK, device=a.device, dtype=torch.float32)
    far = i[:, None] - i[None, :]
    w = torch.where(far >= 0, torch.exp(g[:, None, None] * far.clamp(min=0)), 0.0)
    inside = (a @ b.transpose(-1, -2) * w[:, None]) @ c
    sums = (b * torch.exp(g[:, None, None, None] * (_CHUNK - 1 - i)[:, None])).transpose(-1, -2) @ c
    j = torch.arange(n, device=a.device, dtype=torch.float32)
    back = j[:, None] - 1 - j[None, :]
    w = torch.where(back >= 0, torch.exp(g[:, None, None] * _CHUNK * back.clamp(min=0)), 0.0)
    start = (w @ sums.flatten(3)).unflatten(-1, (X, Y))
    if state is not None:
        start = start + torch.exp(g[:, None] * _CHUNK * j)[..., None, None] * state[:, :, None]
    before = (a @ start) * torch.exp(g[:, None, None] * (i + 1))[..., None]
    return (scale * (inside + before)).flatten(2, 3)[:, :, :T]


def _plain_state(k, v, g, n, state, ahead):
    """sum_{j<n} lam^{n-1-j+ahead} k_j v_j^T (+ lam^n state) with n [B]; k, v are zero from n on."""
    j = torch.arange(k.shape[2], device=k.device, dtype=torch.float32)
    back = (n.float()[:, None] - 1 - j).clamp(min=0) + ahead
    s = (k * torch.exp(g[None, :, None] * back[:, None])[..., None]).transpose(-1, -2) @ v
    return s if state is None else s + torch.exp(g[None, :] * n.float()[:, None])[..., None, None] * state


def _plain_inputs(s, *names):
    """[B, T, H, .] tensors as float32 [B, H, T, .] with zeros from each row's length on, and the lengths."""
    x = s["q"]
    T = x.shape[1]
    n = s["lengths"]
    n = torch.full((x.shape[0],), T, device=x.device, dtype=torch.int32) if n is None else n.clamp(0, T)
    inside = (torch.arange(T, device=x.device) < n[:, None])[:, None, :, None]
    return [torch.where(inside, s[m].transpose(1, 2).float(), 0.0) for m in names], n, inside


def _plain_forward(s):
    (q, k, v), n, _ = _plain_inputs(s, "q", "k", "v")
    out = _plain_scan(q, k, v, s["log_decay"], s["state"], s["scale"])
    return out.transpose(1, 2).to(s["q"].dtype), _plain_state(k, v, s["log_decay"], n, s["state"], 0)


def _plain_backward(s):
    (q, k, v, do), n, inside = _plain_inputs(s, "q", "k", "v", "grad_out")
    g, scale, dt = s["log_decay"], s["scale"], s["q"].dtype
    T = q.shape[2]
    state = s["state"]
    gq = _plain_scan(do, v, k, g, None if state is None else state.transpose(-1, -2), scale)
    # reverse time: position t of a row of length n is its position n - 1 - t
    turn = ((n[:, None] - 1 - torch.arange(T, device=q.device)) % T)[:, None, :, None]

    def rev(x):
        return torch.where(inside, x.gather(2, turn.expand(x.shape).long()), 0.0)

    gs = s["grad_state"]
    start = None if gs is None else gs * torch.exp(-g)[:, None, None] / scale
    q_, k_, v_, do_ = rev(q), rev(k), rev(v), rev(do)
    gk = rev(_plain_scan(v_, do_, q_, g, None if start is None else start.transpose(-1, -2), scale))
    gv = rev(_plain_scan(k_, q_, do_, g, start, scale))
    grads = [x.transpose(1, 2).to(dt) for x in (gq, gk, gv)]
    if gs is None:
        return grads
    return grads + [_plain_state(q_ * scale, do_, g, n, gs, 1)]


def _plain_step(s):
    q, k, v = (s[m].float() for m in ("q", "k", "v"))
    new = torch.exp(s["log_decay"])[:, None, None] * s["state"] + k[..., None] * v[..., None, :]
    y = s["scale"] * (q[..., None, :] @ new)[..., 0, :]
    s["state_out"].copy_(new)
    return y.to(s["q"].dtype), s["state_out"]


def _plain_rotary(s):
    c = s["case"]
    R = c["R"]
    angle = s["positions"].double()[..., None] * s["inv_freq"]
    if c["inverse"]:
        angle = -angle
    cos = (angle.cos() * s["mscale"]).float()[:, :, None]
    sin = (angle.sin() * s["mscale"]).float()[:, :, None]

    def turn(x):
        r = x[..., :R].float()
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = r[..., :R // 2], r[..., R // 2:]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((r.to(x.dtype), x[..., R:]), -1)

    return turn(s["q"]), turn(s["k"])


# -------------------------------------------------------------------- run ---

def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        import rwkv_linear_rnn_b200 as W
        if kind == "rotary":
            return W.linattn_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], mscale=s["mscale"],
                                    interleaved=c["interleaved"], inverse=c["inverse"])
        if kind == "step":
            return W.linattn_decay_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"],
                                        state_out=s["state_out"])
        if kind == "prompt":
            return W.linattn_decay_forward(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"],
                                           lengths=s["lengths"], want_state=True)
        out, _ = W.linattn_decay_forward(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"],
                                         lengths=s["lengths"])
        grads = W.linattn_decay_backward(s["q"], s["k"], s["v"], s["log_decay"], s["grad_out"], s["state"],
                                         scale=s["scale"], lengths=s["lengths"], grad_state_out=s["grad_state"],
                                         want_grad_state=c["state"])
        return [out] + [x for x in grads if x is not None]
    if kind == "rotary":
        return _plain_rotary(s)
    if kind == "step":
        return _plain_step(s)
    if kind == "prompt":
        return _plain_forward(s)
    return [_plain_forward(s)[0]] + _plain_backward(s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T = case["B"], case["T"]
    if case["kind"] == "rotary":
        n = B * T * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * e * n * case["D"] + 8 * B * T, "flops": 3 * n * case["R"]}
    H, D, M = case["H"], case["D"], case["M"]
    tokens, state = B * T * H, 4 * B * H * D * M
    if case["kind"] == "step":
        return {"bytes": e * tokens * 2 * (D + M) + 2 * state, "flops": 5 * tokens * D * M}
    if case["kind"] == "prompt":
        return {"bytes": e * tokens * 2 * (D + M) + state * (2 if case["state"] else 1), "flops": 4 * tokens * D * M}
    return {"bytes": e * tokens * 4 * (D + M) + state * (3 if case["state"] else 0), "flops": 12 * tokens * D * M}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    """The recurrences themselves, one position after the other, in float64; complex products for the rotation."""
    s = prepare(case, seed)
    if case["kind"] == "rotary":
        turn = s["mscale"] * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                         s["positions"].double()[..., None] * s["inv_freq"])
        turn = (turn.conj() if case["inverse"] else turn)[:, :, None]
        out = []
        for x in (s["q"], s["k"]):
            y = x.double()
            if case["interleaved"]:
                at, bt = slice(0, case["R"], 2), slice(1, case["R"], 2)
            else:
                at, bt = slice(0, case["R"] // 2), slice(case["R"] // 2, case["R"])
            z = torch.complex(y[..., at], y[..., bt]) * turn
            y[..., at], y[..., bt] = z.real, z.imag
            out.append(y)
        return out
    lam = s["log_decay"].double().exp()[:, None, None]
    if case["kind"] == "step":
        new = s["state"].double() * lam + torch.einsum("nhd,nhm->nhdm", s["k"].double(), s["v"].double())
        return torch.einsum("nhd,nhdm->nhm", s["q"].double(), new) * s["scale"], new
    q, k, v = s["q"], s["k"], s["v"]
    B, T, H, D = q.shape
    M = v.shape[-1]
    n = s["lengths"]
    live = None if n is None else (torch.arange(T, device="cuda")[:, None] < n).double()[:, :, None, None, None]

    def column(x, t):
        return x[:, t].double().unsqueeze(-1)

    def row(x, t):
        return x[:, t].double().unsqueeze(-2)

    def empty():
        return torch.zeros(B, H, D, M, dtype=torch.float64, device="cuda")

    train = case["kind"] == "train"
    S = empty() if s["state"] is None else s["state"].double()
    out = torch.zeros(B, T, H, M, dtype=torch.float64, device="cuda")
    gq = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda") if train else None
    for t in range(T):
        new = torch.baddbmm((S * lam).flatten(0, 1), column(k, t).flatten(0, 1), row(v, t).flatten(0, 1))
        new = new.unflatten(0, (B, H))
        y = row(q, t) @ new
        if train:
            z = new @ column(s["grad_out"], t)
            gq[:, t] = (z if live is None else z * live[t])[..., 0]
        if live is not None:
            y = y * live[t]
            new = torch.where(live[t] > 0, new, S)
        out[:, t] = y[..., 0, :]
        S = new
    out *= s["scale"]
    if not train:
        return out, S
    gk, gv = torch.zeros_like(gq), torch.zeros_like(out)
    G = empty() if s["grad_state"] is None else s["grad_state"].double()  # the gradient of the state after position t
    for t in range(T - 1, -1, -1):
        X = G + s["scale"] * column(q, t) * row(s["grad_out"], t)
        x, y = X @ column(v, t), row(k, t) @ X
        if live is not None:
            x, y = x * live[t], y * live[t]
            G = torch.where(live[t] > 0, X * lam, G)
        else:
            G = X * lam
        gk[:, t], gv[:, t] = x[..., 0], y[..., 0, :]
    grads = [out, gq * s["scale"], gk, gv]
    return grads if s["grad_state"] is None else grads + [G]
