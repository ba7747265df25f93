"""The operators around the KDA layer, as they are measured: the gated linear recurrence (forward,
gradients, one token), the norms around a block (forward, gradients) and the KDA step of one token.

``run`` computes a case in plain torch operations in 32 bits (``own`` false) or by the library's calls
(``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.

Cases (a dict of plain values):
  op       scan | scan_grad | scan_step | norm | norm_grad | decode
  type     type of the activations: bf16, f16 or f32
scan, scan_grad: T tokens in N packed sequences of ragged lengths, D channels; split: x and i are the two
  halves of one projection's rows (row stride 2 D) instead of tensors of their own; h0: with initial states.
scan_step: B tokens, each the next one of its own slot in a pool of states, D channels.
norm, norm_grad: T rows of D channels; res: type of the residual stream; group: channels of a group of the
  norm after the block (0: the whole row); gate: none, sigmoid or silu; ls: with a per-channel residual scale.
decode: B tokens, each the next one of its own slot, H heads of 128 x 128 states.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
TILE = 128      # tokens between two saved states of the recurrence
K = 128         # key and value width of a KDA head
EPS = 1e-6


def listed():
    return [
        # a short prompt through a narrow layer: launch latency counts
        {"name": "scan_t1024_d512", "op": "scan", "T": 1024, "N": 1, "D": 512, "type": "bf16", "split": False, "h0": False},
        # prefill or training of a packed batch at full width (24 sequences that continue from earlier states)
        {"name": "scan_packed65536_d4096", "op": "scan", "T": 65536, "N": 24, "D": 4096, "type": "bf16", "split": True, "h0": True},
        # odd sizes: lengths and a width that no tile or vector divides, in 32 bits
        {"name": "scan_t5003_d1001_f32", "op": "scan", "T": 5003, "N": 7, "D": 1001, "type": "f32", "split": False, "h0": True},
        # one layer's gradients, one sequence
        {"name": "scan_grad_t8192_d2048", "op": "scan_grad", "T": 8192, "N": 1, "D": 2048, "type": "bf16", "split": False, "h0": True},
        # gradients of a packed batch of ragged documents
        {"name": "scan_grad_packed32768_d4096", "op": "scan_grad", "T": 32768, "N": 61, "D": 4096, "type": "f16", "split": True, "h0": False},
        # one decoding step of a batch of 64
        {"name": "scan_step_b64_d2048", "op": "scan_step", "B": 64, "D": 2048, "type": "bf16"},
        # the norms around a block in a decoding step of 8 tokens
        {"name": "norm_t8_d2048", "op": "norm", "T": 8, "D": 2048, "type": "bf16", "res": "bf16", "group": 0, "gate": "none", "ls": True},
        # the gated head norm of a packed batch, a residual stream in 32 bits
        {"name": "norm_t65536_d4096_heads", "op": "norm", "T": 65536, "D": 4096, "type": "bf16", "res": "f32", "group": 128, "gate": "sigmoid", "ls": False},
        # gradients of the norms of one layer
        {"name": "norm_grad_t8192_d2048", "op": "norm_grad", "T": 8192, "D": 2048, "type": "bf16", "res": "bf16", "group": 128, "gate": "sigmoid", "ls": True},
        # odd sizes, the whole row normed, in 32 bits
        {"name": "norm_grad_t4099_d1001_f32", "op": "norm_grad", "T": 4099, "D": 1001, "type": "f32", "res": "f32", "group": 0, "gate": "silu", "ls": True},
        # a decoding step of two tokens
        {"name": "decode_b2_h16", "op": "decode", "B": 2, "H": 16, "type": "bf16"},
        # a decoding step of a full batch
        {"name": "decode_b256_h32", "op": "decode", "B": 256, "H": 32, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["scan", "scan_grad", "scan_step", "norm", "norm_grad", "decode"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "decode":
        return {"op": op, "B": _log(rng, 1, 250), "H": rng.randint(1, 32), "type": kind}
    # mostly widths that whole heads give, some that nothing divides
    D = rng.choice([1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 28, 32]) * 128 if rng.random() < 0.7 else _log(rng, 33, 4095)
    if op == "scan_step":
        return {"op": op, "B": _log(rng, 1, 2048), "D": D, "type": kind}
    most = 200_000_000 if op in ("scan", "norm") else 110_000_000      # elements
    if kind == "f32":
        most //= 2
    T = min(_log(rng, 1, 65000), most // D)
    if op in ("scan", "scan_grad"):
        return {"op": op, "T": T, "N": min(T, _log(rng, 1, 200)), "D": D, "type": kind, "split": rng.random() < 0.5,
                "h0": rng.random() < 0.5}
    return {"op": op, "T": T, "D": D, "type": kind, "res": rng.choice([kind, "f32"]),
            "group": rng.choice([0, 128]) if D % 128 == 0 else 0, "gate": rng.choice(["none", "sigmoid", "silu"]),
            "ls": rng.random() < 0.5}


def _lengths(T, N, seed):
    """N ragged lengths of one token or more that sum to T, log-uniform over a factor of 32."""
    gen = torch.Generator().manual_seed(seed)
    w = torch.exp(torch.rand(N, generator=gen, dtype=torch.float64) * math.log(32.0))
    n = 1 + torch.floor(w / w.sum() * (T - N)).to(torch.int64)
    n[0] += T - int(n.sum())
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def decay(rows, D):
        # log-decays: every channel has its own time scale, 5 to 1000 tokens, that varies by the token
        scale = torch.exp(torch.empty(D, device="cuda").uniform_(math.log(1e-3), math.log(0.2), generator=gen))
        return -scale * torch.empty(rows, D, device="cuda").uniform_(0.2, 1.8, generator=gen)

    s = dict(case)
    op = case["op"]
    if op in ("scan", "scan_grad"):
        T, N, D = case["T"], case["N"], case["D"]
        n = _lengths(T, N, seed)
        cu = torch.zeros(N + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(n, 0)
        s["cu"], s["longest"] = cu.tolist(), int(n.max())
        s["starts"], s["ends"] = cu[:-1].cuda(), (cu[1:] - 1).cuda()
        if case["split"]:
            xi = normal(T, 2 * D, dtype=t)
            xi[:, D:] = torch.sigmoid(xi[:, D:].float()).to(t)
            s["x"], s["i"] = xi[:, :D], xi[:, D:]
        else:
            s["x"], s["i"] = normal(T, D, dtype=t), torch.sigmoid(normal(T, D)).to(t)
        s["g"] = decay(T, D)
        s["h0"] = normal(N, D) if case["h0"] else None
        if op == "scan_grad":
            s["dh"], s["dfinal"] = normal(T, D, dtype=t), normal(N, D)
            # what the forward saved: the state before every 128th token
            h = _recurrence(s["x"], s["i"], s["g"], s["h0"], s["starts"], s["longest"])
            s["states"] = torch.cat([torch.zeros_like(h[:1]), h[TILE - 1:T - 1:TILE]]).contiguous()
            del h
    elif op == "scan_step":
        B, D = case["B"], case["D"]
        s["x"], s["i"], s["g"] = normal(B, D, dtype=t), torch.sigmoid(normal(B, D)).to(t), decay(B, D)
        s["state"] = normal(B + 3, D)
        s["slots"] = torch.randperm(B + 3, generator=gen, device="cuda")[:B].to(torch.int32)
    elif op == "decode":
        B, H = case["B"], case["H"]
        unit = lambda v: v / torch.linalg.vector_norm(v, dim=-1, keepdim=True)
        s["q"], s["k"] = unit(normal(B, H, K)).to(t), unit(normal(B, H, K)).to(t)
        s["v"], s["beta"] = normal(B, H, K, dtype=t), torch.sigmoid(normal(B, H))
        s["g"] = torch.empty(B, H, K, device="cuda").uniform_(-0.2, -0.001, generator=gen)
        s["state"] = normal(B + 3, H, K, K, std=0.1)
        s["slots"] = torch.randperm(B + 3, generator=gen, device="cuda")[:B].to(torch.int32)
        s["scale"] = K ** -0.5
    else:
        T, D = case["T"], case["D"]
        rt = TYPES[case["res"]]
        G = case["group"] or D
        s["o"] = normal(T, D, dtype=t, std=0.5)
        s["z"] = normal(T, D, dtype=t) if case["gate"] != "none" else None
        s["w_post"], s["w_pre"] = 1 + normal(G, std=0.1), 1 + normal(D, std=0.1)
        s["scale"], s["ls"] = 0.5, (1 + normal(D, std=0.2) if case["ls"] else None)
        s["r"] = normal(T, D, dtype=rt, std=2.0)     # the residual before (forward) or after (gradients) the block
        if op == "norm_grad":
            s["dr"], s["dy"] = normal(T, D, dtype=rt), normal(T, D, dtype=t)
    if own:
        _plan(s, t)
    return s


def _plan(s, t):
    """The plan, workspace and output buffers that a user's program keeps."""
    import context_kda_gb300 as kda
    op = s["op"]
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")
    if op in ("scan", "scan_grad"):
        T, N, D = s["T"], s["N"], s["D"]
        s["plan"] = kda.kda_plan_segments(s["cu"], 1)
        s["plan_dev"] = kda.upload_plan(s["plan"])
        s["ws"] = new(kda.kda_gated_scan_workspace_bytes(s["plan"], D), dtype=torch.uint8)
        if op == "scan":
            s["h"], s["final"] = new(T, D, dtype=t), new(N, D)
        else:
            s["dx"], s["di"], s["dg"], s["dh0"] = new(T, D, dtype=t), new(T, D, dtype=t), new(T, D), new(N, D)
    elif op == "scan_step":
        s["h"] = new(s["B"], s["D"], dtype=t)
    elif op == "decode":
        s["out"] = new(s["B"], s["H"], K, dtype=t)
    else:
        T, D, rt = s["T"], s["D"], s["r"].dtype
        if op == "norm":
            s["r_out"], s["y"] = new(T, D, dtype=rt), new(T, D, dtype=t)
        else:
            s["ws"] = new(kda.kda_block_norm_workspace_bytes(D), dtype=torch.uint8)
            s["dr_in"], s["do"] = new(T, D, dtype=rt), new(T, D, dtype=t)
            s["dz"] = None if s["z"] is None else new(T, D, dtype=t)
            s["dw_post"], s["dw_pre"] = new(s["group"] or D), new(D)
            s["dls"] = None if s["ls"] is None else new(D)


def run(s):
    return (_own if own else _plain)[s["op"]](s)


# ---- the library's calls ----------------------------------------------------------------------------


def _own_scan(s):
    import context_kda_gb300 as kda
    kda.kda_gated_scan_forward(s["plan"], s["plan_dev"], s["x"], s["i"], s["g"], s["h0"], s["h"], s["final"], None, s["ws"])
    return {"h": s["h"], "final": s["final"]}


def _own_scan_grad(s):
    import context_kda_gb300 as kda
    kda.kda_gated_scan_backward(s["plan"], s["plan_dev"], s["x"], s["i"], s["g"], s["h0"], s["states"], s["dh"], s["dfinal"],
                                s["dx"], s["di"], s["dg"], s["dh0"], s["ws"])
    return {"dx": s["dx"], "di": s["di"], "dg": s["dg"], "dh0": s["dh0"]}


def _own_scan_step(s):
    import context_kda_gb300 as kda
    kda.kda_gated_scan_step(s["slots"], s["x"], s["i"], s["g"], s["state"], s["h"])
    return {"h": s["h"], "state": s["state"]}


def _own_norm(s):
    import context_kda_gb300 as kda
    kda.kda_block_norm_forward(s["r"], s["o"], s["z"], s["gate"], s["group"], s["w_post"], s["scale"], s["ls"], s["w_pre"], EPS,
                               s["r_out"], s["y"])
    return {"r": s["r_out"], "y": s["y"]}


def _own_norm_grad(s):
    import context_kda_gb300 as kda
    kda.kda_block_norm_backward(s["r"], s["o"], s["z"], s["gate"], s["group"], s["w_post"], s["scale"], s["ls"], s["w_pre"], EPS,
                                s["dr"], s["dy"], s["dr_in"], s["do"], s["dz"], s["dw_post"], s["dls"], s["dw_pre"], s["ws"])
    return {"dr": s["dr_in"], "do": s["do"], "dz": s["dz"], "dw_post": s["dw_post"], "dls": s["dls"], "dw_pre": s["dw_pre"]}


def _own_decode(s):
    import context_kda_gb300 as kda
    kda.kda_decode_step(s["slots"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["state"], s["out"])
    return {"o": s["out"], "state": s["state"]}


# ---- the plain forms ------------------------------------------------------------------------------------


def _doubling(a, b, longest, dim=0):
    """h_t = a_t h_{t-1} + b_t along `dim` (a_t = 0 where a sequence starts) by doubling: after the step of
    length d every element holds its last 2 d terms.  a and b are overwritten; returns b."""
    d, T = 1, a.shape[dim]
    while d < min(longest, T):
        cur, before = [a.narrow(dim, d, T - d), b.narrow(dim, d, T - d)], [a.narrow(dim, 0, T - d), b.narrow(dim, 0, T - d)]
        new_b = cur[1] + cur[0] * before[1]
        cur[0].copy_(cur[0] * before[0])
        cur[1].copy_(new_b)
        d *= 2
    return b


def _recurrence(x, i, g, h0, starts, longest):
    a, b = torch.exp(g), x.float() * i.float()
    if h0 is not None:
        b[starts] += a[starts] * h0
    a[starts] = 0
    return _doubling(a, b, longest)


def _plain_scan(s):
    h = _recurrence(s["x"], s["i"], s["g"], s["h0"], s["starts"], s["longest"])
    return {"h": h.to(s["x"].dtype), "final": h[s["ends"]]}


def _plain_scan_grad(s):
    x, i, T, D = s["x"].float(), s["i"].float(), s["T"], s["D"]
    starts, ends = s["starts"], s["ends"]
    a = torch.exp(s["g"])
    # the states within every tile of 128 tokens from the one that the forward saved
    tiles = -(-T // TILE)
    w, b = torch.zeros(tiles * TILE, D, device="cuda"), torch.zeros(tiles * TILE, D, device="cuda")
    w[:T], b[:T] = a, x * i
    if s["h0"] is not None:
        b[starts] += a[starts] * s["h0"]
    w[starts] = 0
    w, b = w.view(tiles, TILE, D), b.view(tiles, TILE, D)
    b[:, 0] += w[:, 0] * s["states"]
    h = _doubling(w, b, min(TILE, s["longest"] + 1), dim=1).view(-1, D)[:T]
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[starts] = 0 if s["h0"] is None else s["h0"]
    # the gradients of the states, from the last token to the first
    c, d = torch.zeros_like(a), s["dh"].float()
    if d is s["dh"]:
        d = d.clone()
    c[:-1] = a[1:]
    c[ends] = 0
    d[ends] += s["dfinal"]
    d = _doubling(c.flip(0), d.flip(0), s["longest"]).flip(0)
    kind = s["x"].dtype
    return {"dx": (i * d).to(kind), "di": (x * d).to(kind), "dg": a * before * d, "dh0": a[starts] * d[starts]}


def _plain_scan_step(s):
    slots = s["slots"].long()
    new = torch.exp(s["g"]) * s["state"][slots] + s["x"].float() * s["i"].float()
    s["state"][slots] = new
    return {"h": new.to(s["x"].dtype), "state": s["state"]}


def _plain_decode(s):
    slots, q, k, v = s["slots"].long(), s["q"].float(), s["k"].float(), s["v"].float()
    S = s["state"][slots] * torch.exp(s["g"]).unsqueeze(-1)
    d = s["beta"].unsqueeze(-1) * (v - (S * k.unsqueeze(-1)).sum(-2))
    S = S + k.unsqueeze(-1) * d.unsqueeze(-2)
    s["state"][slots] = S
    return {"o": (s["scale"] * (S * q.unsqueeze(-1)).sum(-2)).to(s["q"].dtype), "state": s["state"]}


def _gate(kind, z):
    """The gate's value and its derivative."""
    if kind == "none":
        return 1.0, 0.0
    p = 1 / (1 + torch.exp(-z))
    return (p, p * (1 - p)) if kind == "sigmoid" else (z * p, p * (1 + z * (1 - p)))


def _unit(v, G):
    """v over the root mean square of its groups of G channels, and the reciprocal of that."""
    w = v.view(v.shape[0], -1, G)
    inv = 1 / torch.sqrt((w * w).mean(-1, keepdim=True) + EPS)
    return (w * inv).view_as(v), inv


def _plain_norm(s):
    T, D = s["T"], s["D"]
    G = s["group"] or D
    act, _ = _gate(s["gate"], None if s["z"] is None else s["z"].float())
    u = act * (_unit(s["o"].float(), G)[0].view(T, -1, G) * s["w_post"]).view(T, D)
    u = s["scale"] * u if s["ls"] is None else s["scale"] * s["ls"] * u
    r = s["r"].float() + u
    y = _unit(r, D)[0] * s["w_pre"]
    return {"r": r.to(s["r"].dtype), "y": y.to(s["o"].dtype)}


def _plain_norm_grad(s):
    T, D = s["T"], s["D"]
    G = s["group"] or D
    kind = s["o"].dtype
    z = None if s["z"] is None else s["z"].float()
    act, slope = _gate(s["gate"], z)
    dy = s["dy"].float()
    r_hat, inv_r = _unit(s["r"].float(), D)
    dw_pre = (dy * r_hat).sum(0)
    e = dy * s["w_pre"]
    dr = s["dr"].float() + inv_r.view(T, 1) * (e - r_hat * (e * r_hat).mean(-1, keepdim=True))
    o_hat, inv_o = _unit(s["o"].float(), G)
    n = (o_hat.view(T, -1, G) * s["w_post"]).view(T, D)
    t = s["scale"] * dr
    dls = None if s["ls"] is None else (t * act * n).sum(0)
    du = t if s["ls"] is None else t * s["ls"]
    dz = None if z is None else (du * n * slope).to(kind)
    dn = du * act
    dw_post = (dn * o_hat).view(T, -1, G).sum((0, 1))
    e = dn.view(T, -1, G) * s["w_post"]
    o_hat = o_hat.view(T, -1, G)
    do = (inv_o * (e - o_hat * (e * o_hat).mean(-1, keepdim=True))).view(T, D)
    return {"dr": dr.to(s["r"].dtype), "do": do.to(kind), "dz": dz, "dw_post": dw_post, "dls": dls, "dw_pre": dw_pre}


_own = {"scan": _own_scan, "scan_grad": _own_scan_grad, "scan_step": _own_scan_step, "norm": _own_norm,
        "norm_grad": _own_norm_grad, "decode": _own_decode}
_plain = {"scan": _plain_scan, "scan_grad": _plain_scan_grad, "scan_step": _plain_scan_step, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad, "decode": _plain_decode}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    return _exact[case["op"]](s, lambda name: wide.get(name))


def _tokens(s, x, i, g, h0):
    """The recurrence token by token, and the state before each token."""
    b, a = (x * i).unbind(0), torch.exp(g).unbind(0)
    h, before = [], []
    for n in range(s["N"]):
        p = torch.zeros_like(a[0]) if h0 is None else h0[n]
        for t in range(s["cu"][n], s["cu"][n + 1]):
            before.append(p)
            p = torch.addcmul(b[t], a[t], p)
            h.append(p)
    return h, before


def _exact_scan(s, w):
    h, _ = _tokens(s, w("x"), w("i"), w("g"), w("h0"))
    final = torch.stack([h[e - 1] for e in s["cu"][1:]])
    return {"h": torch.stack(h), "final": final}


def _exact_scan_grad(s, w):
    x, i, g = w("x"), w("i"), w("g")
    before = torch.stack(_tokens(s, x, i, g, w("h0"))[1])
    a, dh = torch.exp(g), w("dh").unbind(0)
    rows, grads, dh0 = a.unbind(0), [None] * s["T"], [None] * s["N"]
    for n in range(s["N"]):
        p = w("dfinal")[n]
        for t in range(s["cu"][n + 1] - 1, s["cu"][n] - 1, -1):
            grads[t] = dh[t] + p
            p = rows[t] * grads[t]
        dh0[n] = p
    d = torch.stack(grads)
    return {"dx": i * d, "di": x * d, "dg": a * before * d, "dh0": torch.stack(dh0)}


def _exact_scan_step(s, w):
    state, slots = w("state").clone(), s["slots"].long()
    state[slots] = torch.exp(w("g")) * state[slots] + w("x") * w("i")
    return {"h": state[slots], "state": state}


def _exact_decode(s, w):
    state, slots = w("state").clone(), s["slots"].long()
    out = torch.empty_like(w("v"))
    for b, slot in enumerate(slots.tolist()):
        S = torch.exp(w("g")[b]).unsqueeze(-1) * state[slot]
        k = w("k")[b]
        d = w("beta")[b].unsqueeze(-1) * (w("v")[b] - torch.einsum("hk,hkv->hv", k, S))
        S = S + torch.einsum("hk,hv->hkv", k, d)
        out[b] = s["scale"] * torch.einsum("hk,hkv->hv", w("q")[b], S)
        state[slot] = S
    return {"o": out, "state": state}


def _exact_parts(s, w):
    """The block's branch, from its definition: the groups' root mean squares, the gate, the scale."""
    T, D = s["T"], s["D"]
    G = s["group"] or D
    o = w("o").reshape(T, D // G, G)
    norm = torch.sqrt(o.pow(2).sum(-1, keepdim=True) / G + EPS)
    post = w("w_post").expand(D // G, G)
    p = None if s["z"] is None else torch.sigmoid(w("z"))
    act = None if p is None else p if s["gate"] == "sigmoid" else w("z") * p
    n = (o / norm * post).reshape(T, D)
    return n, act, p, o / norm, norm, post


def _exact_norm(s, w):
    n, act, _, _, _, _ = _exact_parts(s, w)
    u = s["scale"] * (n if act is None else n * act)
    r = w("r") + (u if s["ls"] is None else u * w("ls"))
    y = r / torch.sqrt(r.pow(2).sum(-1, keepdim=True) / s["D"] + EPS) * w("w_pre")
    return {"r": r, "y": y}


def _exact_norm_grad(s, w):
    T, D = s["T"], s["D"]
    n, act, p, hat, norm, post = _exact_parts(s, w)
    G = hat.shape[-1]
    r, dy = w("r"), w("dy")
    size = torch.sqrt(r.pow(2).sum(-1, keepdim=True) / D + EPS)
    e = dy * w("w_pre")
    dr = w("dr") + e / size - r * (e * r).sum(-1, keepdim=True) / (D * size.pow(3))
    t = s["scale"] * dr
    u = n if act is None else n * act
    dls = None if s["ls"] is None else (t * u).sum(0)
    if s["ls"] is not None:
        t = t * w("ls")
    dz = None
    if act is not None:
        slope = p * (1 - p) if s["gate"] == "sigmoid" else p + w("z") * p * (1 - p)
        dz = t * n * slope
        t = t * act
    t = t.reshape(T, D // G, G)
    dw_post = (t * hat).sum((0, 1))
    t = t * post
    do = ((t - hat * (t * hat).sum(-1, keepdim=True) / G) / norm).reshape(T, D)
    return {"dr": dr, "do": do, "dz": dz, "dw_post": dw_post, "dls": dls, "dw_pre": (dy * r / size).sum(0)}


_exact = {"scan": _exact_scan, "scan_grad": _exact_scan_grad, "scan_step": _exact_scan_step, "norm": _exact_norm,
          "norm_grad": _exact_norm_grad, "decode": _exact_decode}


def work(case):
    """Bytes: every input once, every output once.  Operations: an exponential counts as one."""
    op, e = case["op"], BYTES[case["type"]]
    if op in ("scan", "scan_grad"):
        n, N, D = case["T"] * case["D"], case["N"], case["D"]
        ends = N * D * 4 * (2 if case["h0"] else 1)                  # final states or dfinal, h0
        if op == "scan":
            return {"bytes": n * (3 * e + 4) + ends, "flops": n * 4}
        return {"bytes": n * (5 * e + 8) + ends + N * D * 4 + -(-case["T"] // TILE) * D * 4, "flops": n * 10}
    if op == "scan_step":
        n = case["B"] * case["D"]
        return {"bytes": n * (3 * e + 12), "flops": n * 4}
    if op == "decode":
        n = case["B"] * case["H"]
        return {"bytes": n * (K * K * 8 + K * (4 * e + 4) + 4), "flops": n * K * K * 7}
    n, D, r = case["T"] * case["D"], case["D"], BYTES[case["res"]]
    gated, G = case["gate"] != "none", case["group"] or case["D"]
    weights = (G + D * (2 if case["ls"] else 1)) * 4
    if op == "norm":
        return {"bytes": n * (2 * r + (3 if gated else 2) * e) + weights, "flops": n * 12}
    return {"bytes": n * (3 * r + (5 if gated else 3) * e) + 2 * weights, "flops": n * 30}
