"""Measured cases of what stands around and behind the Mamba-2 scan: the short
causal convolution in front of it, the scan's gradients, and the RMS norm with
the residual's addition between blocks; with their plain forms in elementary
torch operations.

`run` computes the plain form where `own` is false and calls the package where
it is true; `exact` evaluates the definitions in 64 bits: the convolution and
the norm through autograd, the scan token by token.
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64  # chunk length of the scan's plain form
_FP8_MAX = 448.0  # the largest value of float8_e4m3fn


# --------------------------------------------------------------- the cases

def listed():
    return [
        # a batch of prompts (or a training step's forward): the scan's x, B
        # and C as columns of the layer's projection, left as three tensors
        _conv("conv_prompt_bf16", "fwd", 8, 2048, 1792, 4, "bf16", fused=True, keep=True, parts=(1536, 128, 128)),
        # documents packed into rows on top of a kept state, odd sizes
        _conv("conv_packed_f32", "fwd", 2, 4133, 1001, 4, "f32", packed=True, state=True, keep=True),
        # gradients of the training step of the first case
        _conv("conv_train_bf16", "bwd", 8, 2048, 1792, 4, "bf16", fused=True, parts=(1536, 128, 128)),
        # gradients over packed documents, with a carried state and its gradient, three taps
        _conv("conv_train_packed_f32", "bwd", 2, 1501, 1000, 3, "f32", packed=True, state=True),
        # one token for each of 256 conversations
        _conv("conv_decode_bf16", "step", 256, 1, 1792, 4, "bf16", state=True, parts=(1536, 128, 128)),
        # gradients of a training step; x, B and C are columns of the convolution's output
        _ssd("ssd_train_bf16", 8, 2048, 24, 1, 128, "bf16", fused=True),
        # gradients over packed documents in float32, a carried state, odd length
        _ssd("ssd_train_packed_f32", 2, 1501, 12, 3, 64, "f32", packed=True, state=True),
        # one long document, trained on in one go
        _ssd("ssd_train_long_bf16", 1, 16384, 24, 1, 128, "bf16"),
        # a training step's norm in front of a block, the residual kept in float32
        _norm("norm_train_bf16", "fwd", 16384, 768, "bf16", "f32"),
        # its gradients
        _norm("norm_train_grads_bf16", "bwd", 16384, 768, "bf16", "f32"),
        # a prompt's norm for an 8-bit projection, scales for blocks of channels
        _norm("norm_fp8_bf16", "fp8", 4096, 2048, "bf16", "bf16", block=128),
        # one token of a few conversations, odd sizes
        _norm("norm_decode_f32", "fwd", 5, 1000, "f32", "f32"),
    ]


def _conv(name, way, batch, seqlen, channels, taps, dtype, packed=False, state=False, keep=False, fused=False, parts=(),
          act="silu", bias=True):
    c = dict(op="conv", way=way, batch=batch, seqlen=seqlen, channels=channels, taps=taps, dtype=dtype, packed=packed,
             state=state, keep=keep, fused=fused, parts=",".join(map(str, parts)), act=act, bias=bias)
    return dict(c, name=name) if name else c


def _ssd(name, batch, seqlen, heads, groups, d_state, dtype, packed=False, state=False, fused=False):
    c = dict(op="ssd", way="bwd", batch=batch, seqlen=seqlen, heads=heads, groups=groups, d_state=d_state, dtype=dtype,
             packed=packed, state=state, fused=fused)
    return dict(c, name=name) if name else c


def _norm(name, way, rows, channels, dtype, residual, block=0):
    c = dict(op="norm", way=way, rows=rows, channels=channels, dtype=dtype, residual=residual, block=block)
    return dict(c, name=name) if name else c


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["conv", "ssd", "ssd", "norm"])
    less = 2 if dtype == "f32" else 1
    if op == "norm":
        way = rng.choice(["fwd", "bwd", "fp8"])
        while True:
            rows, channels = _spread(rng, 1, 40000), _spread(rng, 33, 16000)
            if way == "fp8" or rng.random() < 0.5:
                channels = (channels + 15) // 16 * 16
            if rows * channels <= 16384 * 768 // less:
                break
        return _norm(None, way, rows, channels, dtype, "f32" if dtype == "f32" else rng.choice(["f32", "bf16"]),
                     block=rng.choice([0, 128]) if way == "fp8" else 0)
    if op == "conv":
        way = rng.choice(["fwd", "bwd", "step"])
        while True:
            batch, seqlen, channels = _spread(rng, 1, 64), _spread(rng, 1, 20000), _spread(rng, 30, 4000)
            if way == "step":
                batch, seqlen = _spread(rng, 1, 512), 1
            if rng.random() < 0.7:
                channels = (channels + 7) // 8 * 8
            if batch * seqlen * channels <= 16384 * 1792 // less:
                break
        parts = ()
        if rng.random() < 0.5:
            side = 8 * max(1, channels // 64)
            parts = (channels - 2 * side, side, side) if channels > 2 * side else ()
        return _conv(None, way, batch, seqlen, channels, rng.choice([2, 3, 4, 4]), dtype,
                     packed=way != "step" and rng.random() < 0.35, state=way == "step" or rng.random() < 0.4,
                     keep=way == "fwd" and rng.random() < 0.6, fused=rng.random() < 0.4, parts=parts,
                     act=rng.choice(["silu", "silu", "none"]), bias=rng.random() < 0.8)
    groups = rng.choice([1, 1, 2, 3, 4])
    heads = groups * rng.choice([1, 2, 3, 8, 24])
    d_state = rng.choice([64, 128])
    while True:
        batch, seqlen = rng.randint(1, 8), _spread(rng, 1, 16000)
        if batch * seqlen * heads * d_state <= 16384 * 24 * 128 // (4 if dtype == "f32" else 1):
            break
    return _ssd(None, batch, seqlen, heads, groups, d_state, dtype, packed=rng.random() < 0.35, state=rng.random() < 0.4,
                fused=rng.random() < 0.5)


# -------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, device="cuda", generator=gen)

    def documents(b, L):  # of about 300 tokens
        first = torch.rand(b, L, device="cuda", generator=gen) < 1 / 300
        return torch.cumsum(first, 1).to(torch.int32)

    t = _DTYPE[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "norm":
        r, c, rt = case["rows"], case["channels"], _DTYPE[case["residual"]]
        spread = torch.exp(0.5 * normal(c))  # channels of different scale
        s["weight"] = 1 + 0.2 * normal(c)
        if case["way"] == "bwd":
            s["h"], s["dy"], s["dh"] = (2 * normal(r, c) * spread).to(rt), normal(r, c, dtype=t), normal(r, c, dtype=rt)
        else:
            s["x"], s["residual"] = normal(r, c, dtype=t), (2 * normal(r, c) * spread).to(rt)
        return s
    b, L = case["batch"], case["seqlen"]
    s["seq_idx"] = documents(b, L) if case["packed"] else None
    if case["op"] == "conv":
        c, k = case["channels"], case["taps"]
        s["weight"] = uniform(-0.5, 0.5, c, k)
        s["bias"] = 0.1 * normal(c) if case["bias"] else None
        if case["fused"]:  # between the gate and dt in the projection's output
            s["x"] = normal(b, L, 2 * c + 24, dtype=t)[..., c:2 * c]
        else:
            s["x"] = normal(b, L, c, dtype=t)
        s["state"] = normal(b, c, k - 1) if case["state"] else None
        parts = [int(p) for p in case["parts"].split(",")] if case["parts"] else None
        s["parts"] = parts
        if case["way"] == "step":
            s["x"] = s["x"][:, 0]
        if case["way"] == "bwd":
            s["dy"] = [normal(b, L, p, dtype=t) for p in parts] if parts else normal(b, L, c, dtype=t)
            s["dstate"] = normal(b, c, k - 1) if case["state"] else None
        return s
    h, g, n = case["heads"], case["groups"], case["d_state"]
    s["A"] = -uniform(1.0, 16.0, h)
    dt = torch.exp(uniform(math.log(1e-3), math.log(1e-1), h))
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))  # softplus of it is dt
    s["D"] = 1 + 0.5 * normal(h)
    if case["fused"]:
        xbc = normal(b, L, h * 64 + 2 * g * n, dtype=t)
        s["x"] = xbc[..., :h * 64].unflatten(-1, (h, 64))
        s["B"] = xbc[..., h * 64:h * 64 + g * n].unflatten(-1, (g, n))
        s["C"] = xbc[..., h * 64 + g * n:].unflatten(-1, (g, n))
        s["dt"] = normal(b, L, 128 + h, dtype=t, scale=0.1)[..., 128:]
    else:
        s["x"], s["B"], s["C"] = normal(b, L, h, 64, dtype=t), normal(b, L, g, n, dtype=t), normal(b, L, g, n, dtype=t)
        s["dt"] = normal(b, L, h, dtype=t, scale=0.1)
    s["dy"] = normal(b, L, h, 64, dtype=t)
    s["state"] = normal(b, h, 64, n) if case["state"] else None
    s["dstate"] = normal(b, h, 64, n) if case["state"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] == "norm":
        return {"fwd": _plain_norm, "fp8": _plain_norm_fp8, "bwd": _plain_norm_grads}[c["way"]](c, state)
    if c["op"] == "conv":
        return _plain_conv_grads(c, state) if c["way"] == "bwd" else _plain_conv(c, state)
    return _plain_ssd_grads(c, state)


def _run_own(c, s):
    import selective_state_space_07_amd as ms
    if c["op"] == "norm":
        if c["way"] == "fwd":
            y, h = ms.add_rms_norm_fwd(s["x"], s["residual"], s["weight"])
            return {"y": y, "h": h}
        if c["way"] == "fp8":
            y, scale, h = ms.add_rms_norm_fp8(s["x"], s["residual"], s["weight"], block=c["block"] or None)
            return {"y": y, "scale": scale, "h": h}
        return ms.add_rms_norm_bwd(s["h"], s["weight"], s["dy"], s["dh"])
    if c["op"] == "conv":
        if c["way"] == "bwd":
            return ms.conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], s["state"], s["dstate"], activation=c["act"],
                               seq_idx=s["seq_idx"])
        if c["way"] == "step":
            y, last = ms.conv_step(s["x"], s["weight"], s["bias"], s["state"], activation=c["act"], split=s["parts"])
        else:
            y, last = ms.conv_fwd(s["x"], s["weight"], s["bias"], s["state"], activation=c["act"], split=s["parts"],
                                  seq_idx=s["seq_idx"], return_state=c["keep"])
        return {"y": y, "state": last} if c["keep"] or c["way"] == "step" else {"y": y}
    return ms.ssd_bwd(s["x"], s["dt"], s["B"], s["C"], s["dt_bias"], s["A"], s["D"], s["dy"], s["state"], s["dstate"],
                      seq_idx=s["seq_idx"])


def _documents(seq_idx, b, L):
    """The number of the document that each token is in, from 0."""
    doc = torch.zeros(b, L, dtype=torch.int64, device="cuda")
    if seq_idx is not None:
        doc[:, 1:] = torch.cumsum((seq_idx[:, 1:] != seq_idx[:, :-1]).long(), 1)
    return doc


# ---------------------------------------------- plain convolution, 32 bits

def _act_grad(name, u):
    s = torch.sigmoid(u)
    return s * (1 + u * (1 - s)) if name == "silu" else torch.ones_like(u)


def _windows(c, s, x, doc):
    """The taps' inputs of each token [taps][b, L, channels], 0 where they are of another document, and the history with x
    behind it."""
    b, L, k = c["batch"], c["seqlen"], c["taps"]
    past = x.new_zeros(b, k - 1, c["channels"]) if s["state"] is None else s["state"].transpose(1, 2)
    wide = torch.cat([past, x], 1)
    docs = torch.cat([doc[:, :1].expand(b, k - 1), doc], 1)
    same = [(docs[:, j:j + L] == doc).unsqueeze(-1) for j in range(k)]
    return [torch.where(same[j], wide[:, j:j + L], 0.0) for j in range(k)], same, wide, docs


def _plain_conv(c, s):
    k, step = c["taps"], c["way"] == "step"
    x = (s["x"].unsqueeze(1) if step else s["x"]).float()
    doc = _documents(s["seq_idx"], c["batch"], c["seqlen"])
    taps, _, wide, docs = _windows(c, s, x, doc)
    u = sum(s["weight"][:, j] * taps[j] for j in range(k))
    if s["bias"] is not None:
        u = u + s["bias"]
    y = (u * torch.sigmoid(u) if c["act"] == "silu" else u).to(s["x"].dtype)
    y = y[:, 0] if step else y
    y = [p.contiguous() for p in y.split(s["parts"], -1)] if s["parts"] else y
    if not c["keep"] and not step:
        return {"y": y}
    last = torch.where((docs[:, -(k - 1):] == doc[:, -1:]).unsqueeze(-1), wide[:, -(k - 1):], 0.0)
    return {"y": y, "state": last.transpose(1, 2).contiguous()}


def _plain_conv_grads(c, s):
    b, L, k = c["batch"], c["seqlen"], c["taps"]
    x, dy = s["x"].float(), (torch.cat(s["dy"], -1) if s["parts"] else s["dy"]).float()
    doc = _documents(s["seq_idx"], b, L)
    taps, same, wide, docs = _windows(c, s, x, doc)
    u = sum(s["weight"][:, j] * taps[j] for j in range(k))
    du = dy * _act_grad(c["act"], u if s["bias"] is None else u + s["bias"])
    got = {"dweight": torch.stack([(du * taps[j]).sum((0, 1)) for j in range(k)], 1)}
    if s["bias"] is not None:
        got["dbias"] = du.sum((0, 1))
    pad = torch.nn.functional.pad
    dwide = sum(pad(torch.where(same[j], s["weight"][:, j] * du, 0.0), (0, 0, j, k - 1 - j)) for j in range(k))
    if s["dstate"] is not None:
        keep = (docs[:, -(k - 1):] == doc[:, -1:]).unsqueeze(-1)
        dwide = dwide + pad(torch.where(keep, s["dstate"].transpose(1, 2), 0.0), (0, 0, L, 0))
    got["dx"] = dwide[:, k - 1:].to(s["x"].dtype).contiguous()
    if s["state"] is not None:
        got["dstate"] = dwide[:, :k - 1].transpose(1, 2).contiguous()
    return got


# ------------------- plain gradients of the scan, in chunks, 32 bits; sums
# ------------------- of step sizes, and what is taken of them, in 64

def _plain_ssd_grads(c, s):
    b, L, h, g, n = (c[k] for k in ("batch", "seqlen", "heads", "groups", "d_state"))
    C = _CHUNK
    m = -(-L // C)
    pad = m * C - L

    def chunks(t):  # [b, L, h or g, d] -> [b, h, m, C, d]
        t = t.float().repeat_interleave(h // t.shape[2], 2).transpose(1, 2)
        return torch.nn.functional.pad(t, (0, 0, 0, pad)).view(b, h, m, C, -1)

    x, Bm, Cm, dy = (chunks(s[k]) for k in ("x", "B", "C", "dy"))
    v = s["dt"].float() + s["dt_bias"]
    delta = torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))
    delta = torch.nn.functional.pad(delta.transpose(1, 2), (0, pad)).view(b, h, m, C)
    A = s["A"].view(1, h, 1, 1)
    cs = torch.cumsum((delta.double() * A.double()).view(b, h, m * C), -1).view(b, h, m, C)
    zero = torch.zeros(b, h, 1, dtype=torch.float64, device="cuda")
    end = cs[..., -1]                                   # behind each chunk
    start = torch.cat([zero, end[..., :-1]], -1)        # before it
    doc = _documents(s["seq_idx"], b, L)
    doc = torch.cat([doc, doc[:, -1:].expand(b, pad)], 1).view(b, 1, m, C)
    last_doc = doc[..., -1]
    open_doc = torch.cat([doc[:, :, :1, 0], last_doc[..., :-1]], -1)  # open where a chunk starts

    def e(t):
        return torch.exp(t).float()

    # inside a chunk
    at = torch.arange(C, device="cuda")
    seen = (doc[..., :, None] == doc[..., None, :]) & (at[:, None] >= at[None, :])
    W = e(torch.where(seen, cs[..., :, None] - cs[..., None, :], -math.inf))
    H = (dy @ x.transpose(-1, -2)) * W                  # [.., r, s]
    G = (Cm @ Bm.transpose(-1, -2)) * W
    d1 = delta[..., None]
    dC = (H * delta[..., None, :]) @ Bm
    dB = d1 * (H.transpose(-1, -2) @ Cm)
    dxi = G.transpose(-1, -2) @ dy                      # dx without delta and D
    M = torch.where(at[:, None] > at[None, :], H * (Cm @ Bm.transpose(-1, -2)) * delta[..., None, :], 0.0).double()
    row, col = M.sum(-1), M.sum(-2)
    inner = torch.flip(torch.cumsum(torch.flip(row - col, (-1,)), -1), (-1,))

    # the state before each chunk and the gradient behind it
    w_own = e(torch.where(doc == last_doc[..., None], end[..., None] - cs, -math.inf)) * delta
    own_S = (x * w_own[..., None]).transpose(-1, -2) @ Bm          # [b, h, m, 64, n]
    w_back = e(torch.where(doc == open_doc[..., None], cs - start[..., None], -math.inf))
    own_R = (dy * w_back[..., None]).transpose(-1, -2) @ Cm
    i = torch.arange(m, device="cuda")
    before = (i[:, None] > i[None, :]) & (open_doc[..., :, None] == last_doc[..., None, :])
    S = (e(torch.where(before, start[..., :, None] - end[..., None, :], -math.inf)) @ own_S.flatten(-2)).view_as(own_S)
    R = (e(torch.where(before.transpose(-1, -2), start[..., None, :] - end[..., :, None], -math.inf)) @ own_R.flatten(-2)).view_as(own_R)
    if s["state"] is not None:
        w = e(torch.where(open_doc == doc[:, :, 0, :1], start, -math.inf))
        S = S + w[..., None, None] * s["state"][:, :, None]
    if s["dstate"] is not None:
        w = e(torch.where(last_doc == doc[:, :, -1, -1:], end[..., -1:] - end, -math.inf))
        R = R + w[..., None, None] * s["dstate"][:, :, None]
    from_S = w_back[..., None] * (dy @ S)
    from_R = e(torch.where(doc == last_doc[..., None], end[..., None] - cs, -math.inf))[..., None]
    dC = dC + from_S
    more = from_R * (Bm @ R.transpose(-1, -2))
    dxi = dxi + more
    dB = dB + d1 * from_R * (x @ R)
    # the gradient of each step's decay exponent
    rows = (from_S * Cm).sum(-1).double()
    cols = (delta * (more * x).sum(-1)).double()
    whole = torch.where(open_doc == last_doc, torch.exp(end - start), 0.0) * (S * R).sum((-1, -2)).double()
    grad = inner + torch.flip(torch.cumsum(torch.flip(rows, (-1,)), -1), (-1,)) + torch.cumsum(cols, -1) - cols + whole[..., None]

    ddelta = (dxi * x).sum(-1) + (A * grad).float()

    def flat(t):  # [b, h, m, C, ..] -> [b, L, h, ..]
        return t.reshape(b, h, m * C, *t.shape[4:])[:, :, :L].transpose(1, 2)

    ddt = flat(ddelta) * torch.sigmoid(v)
    dyf, xf = s["dy"].float(), s["x"].float()
    t = s["x"].dtype
    got = {"dx": (flat(dxi * d1) + s["D"].view(1, 1, h, 1) * dyf).to(t), "ddt": ddt.to(t),
           "dB": flat(dB).unflatten(2, (g, h // g)).sum(3).to(t), "dC": flat(dC).unflatten(2, (g, h // g)).sum(3).to(t),
           "ddt_bias": ddt.sum((0, 1)), "dA": (grad * delta).sum((0, 2, 3)).float(), "dD": (dyf * xf).sum((0, 1, 3))}
    if s["state"] is not None:
        w = e(torch.where(doc[:, :, 0, 0] == last_doc[..., 0], end[..., 0], -math.inf))
        got["dstate"] = own_R[:, :, 0] + w[..., None, None] * R[:, :, 0]
    return got


# -------------------------------------------------- plain norm, 32 bits

def _normed(h):
    return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5)


def _plain_norm(c, s):
    h = s["x"].float() + s["residual"].float()
    return {"y": (_normed(h) * s["weight"]).to(s["x"].dtype), "h": h.to(s["residual"].dtype)}


def _plain_norm_fp8(c, s):
    h = s["x"].float() + s["residual"].float()
    y = _normed(h) * s["weight"]
    r, n = y.shape
    block = c["block"] or n
    wide = torch.nn.functional.pad(y, (0, -n % block)).view(r, -1, block)
    most = wide.abs().amax(-1)
    scale = torch.where(most > 0, most / _FP8_MAX, 1.0)
    q = (wide / scale[..., None]).view(r, -1)[:, :n]
    return {"y": q.to(torch.float8_e4m3fn), "scale": scale, "h": h.to(s["residual"].dtype)}


def _plain_norm_grads(c, s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5)
    hat, dn = h * r, dy * s["weight"]
    d = s["dh"].float() + r * (dn - hat * (dn * hat).mean(-1, keepdim=True))
    return {"dx": d.to(s["dy"].dtype), "dresidual": d.to(s["h"].dtype), "dweight": (dy * hat).sum(0)}


# ----------------------------------------------------------- what it costs

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, r = case["rows"] * case["channels"], 2 if case["residual"] == "bf16" else 4
        if case["way"] == "bwd":
            same = case["dtype"] == case["residual"]
            return {"bytes": n * (e + 2 * r + r + (0 if same else e)) + 8 * case["channels"], "flops": 12 * n}
        out = e if case["way"] == "fwd" else 1
        scales = 4 * case["rows"] * (-(-case["channels"] // case["block"]) if case["block"] else 1)
        return {"bytes": n * (e + 2 * r + out) + 4 * case["channels"] + (scales if case["way"] == "fp8" else 0),
                "flops": 6 * n}
    b, L = case["batch"], case["seqlen"]
    ids = 4 * b * L if case["packed"] else 0
    if case["op"] == "conv":
        c, k = case["channels"], case["taps"]
        n, st, par = b * L * c, 4 * b * c * (k - 1), 4 * c * (k + int(case["bias"]))
        if case["way"] == "bwd":
            return {"bytes": 3 * n * e + ids + 2 * par + 3 * st * int(case["state"]), "flops": n * (6 * k + 8)}
        return {"bytes": 2 * n * e + ids + par + st * (int(case["state"]) + int(case["keep"] or case["way"] == "step")),
                "flops": n * (2 * k + 4)}
    h, g, n = case["heads"], case["groups"], case["d_state"]
    xs, bc, st = b * L * h * 64 * e, b * L * g * n * e, b * h * 64 * n * 4
    # one multiply-add of every state element for every token, in each of the five products that the gradients are
    return {"bytes": 3 * xs + 4 * bc + 2 * b * L * h * e + ids + 3 * st * int(case["state"]) + 24 * h,
            "flops": 10 * b * L * h * 64 * n}


# -------------------------------------------------------- 64 bits, elsewhere

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "ssd": _exact_ssd}[case["op"]](case, s)


def _exact_norm(case, s):
    w = s["weight"].double().requires_grad_(True)
    h = (s["h"].double() if case["way"] == "bwd" else s["x"].double() + s["residual"].double()).requires_grad_(True)
    y = h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + 1e-5) * w
    if case["way"] == "fwd":
        return {"y": y.detach(), "h": h.detach()}
    if case["way"] == "bwd":
        dh, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        return {"dx": dh + s["dh"].double(), "dresidual": dh + s["dh"].double(), "dweight": dw}
    y = y.detach()
    blocks = y.split(case["block"], -1) if case["block"] else [y]
    scale = torch.stack([p.abs().amax(-1) / 448 for p in blocks], -1)
    q = torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(blocks)], -1)
    return {"y": q, "scale": scale, "h": h.detach()}


def _exact_conv(case, s):
    b, L, c, k = (case[n] for n in ("batch", "seqlen", "channels", "taps"))
    leaves = {n: s[n].double().detach().requires_grad_(True) for n in ("x", "weight", "bias", "state") if s[n] is not None}
    x = leaves["x"].view(b, L, c) if case["way"] != "step" else leaves["x"].unsqueeze(1)
    past = leaves["state"].transpose(1, 2) if "state" in leaves else torch.zeros(b, k - 1, c, dtype=torch.float64, device="cuda")
    # how many tokens of its own document stand before each token (the incoming state's count as the first one's)
    age = torch.full((b, L), k, dtype=torch.int64, device="cuda")
    if s["seq_idx"] is not None:
        begins = torch.zeros(b, L, dtype=torch.bool, device="cuda")
        begins[:, 1:] = s["seq_idx"][:, 1:] != s["seq_idx"][:, :-1]
        place = torch.arange(L, device="cuda").expand(b, L)
        newest = torch.cummax(torch.where(begins, place, -1), 1).values
        age = torch.where(newest >= 0, place - newest, k)
    line = torch.cat([past, x], 1)
    u = torch.zeros(b, L, c, dtype=torch.float64, device="cuda")
    for back in range(k):
        u = u + torch.where((age >= back)[..., None], line[:, k - 1 - back:k - 1 - back + L], 0.0) * leaves["weight"][:, k - 1 - back]
    u = u + leaves["bias"] if "bias" in leaves else u
    y = torch.nn.functional.silu(u) if case["act"] == "silu" else u
    # entry i of the state behind the last token is k - 2 - i tokens before it
    keep = torch.arange(k - 2, -1, -1, device="cuda") <= age[:, -1:]
    last = torch.where(keep[..., None], line[:, L:], 0.0).transpose(1, 2)
    if case["way"] == "bwd":
        dy = torch.cat(s["dy"], -1) if case["parts"] else s["dy"]
        out, grad = [y], [dy.double()]
        if s["dstate"] is not None:
            out, grad = out + [last], grad + [s["dstate"].double()]
        grads = torch.autograd.grad(out, list(leaves.values()), grad)
        return {"d" + n: t for n, t in zip(leaves, grads)}
    y, last = y.detach(), last.detach()
    y = y[:, 0] if case["way"] == "step" else y
    y = list(y.split(s["parts"], -1)) if s["parts"] else y
    return {"y": y, "state": last} if case["keep"] or case["way"] == "step" else {"y": y}


def _exact_ssd(case, s):
    b, L, h, g, n = (case[k] for k in ("batch", "seqlen", "heads", "groups", "d_state"))
    rep = h // g
    x, dy = (s[k].double().transpose(0, 1).contiguous() for k in ("x", "dy"))
    Bm, Cm = (s[k].double().repeat_interleave(rep, 2).transpose(0, 1).contiguous() for k in ("B", "C"))
    v = (s["dt"].double() + s["dt_bias"].double()).transpose(0, 1)
    delta = torch.nn.functional.softplus(v, threshold=60)
    same = torch.ones(L, b, 1, dtype=torch.float64, device="cuda")
    if s["seq_idx"] is not None:
        same[1:, :, 0] = (s["seq_idx"][:, 1:] == s["seq_idx"][:, :-1]).double().t()
    keep = torch.exp(delta * s["A"].double()) * same  # the factor on the state before each token
    S = torch.zeros(b, h, 64, n, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    dC, ys = [], []
    for t in range(L):
        S = torch.addcmul(S * keep[t][..., None, None], (delta[t][..., None] * x[t])[..., None], Bm[t].unsqueeze(-2))
        dC.append((dy[t].unsqueeze(-2) @ S).squeeze(-2))
        ys.append((dC[t] * Cm[t]).sum(-1))
    R = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    run = (R * S).sum((-1, -2))  # of the exponent behind the token: <R, decayed S>
    dB, dx, dd, dlog = [None] * L, [None] * L, [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        R = torch.addcmul(R, dy[t][..., None], Cm[t].unsqueeze(-2))
        dB[t] = delta[t][..., None] * (x[t].unsqueeze(-2) @ R).squeeze(-2)
        rb = (R @ Bm[t].unsqueeze(-1)).squeeze(-1)
        dx[t] = delta[t][..., None] * rb
        dd[t] = (rb * x[t]).sum(-1)
        # <R_t, S_t> is what came back from behind plus this token's output; its own input's share is not of the decay
        run = (run + ys[t] - delta[t] * dd[t]) * same[t]
        dlog[t] = run
        R = R * keep[t][..., None, None]
    dlog = torch.stack(dlog)
    ddt = (torch.stack(dd) + s["A"].double() * dlog) * torch.sigmoid(v)

    def heads(t):  # [L, b, h, n] -> [b, L, g, n]
        return torch.stack(t).transpose(0, 1).unflatten(2, (g, rep)).sum(3)

    got = {"dx": (torch.stack(dx) + s["D"].double().view(1, 1, h, 1) * dy).transpose(0, 1), "ddt": ddt.transpose(0, 1),
           "dB": heads(dB), "dC": heads(dC), "ddt_bias": ddt.sum((0, 1)), "dA": (dlog * delta).sum((0, 1)),
           "dD": (dy * x).sum((0, 1, 3))}
    return dict(got, dstate=R) if s["state"] is not None else got
