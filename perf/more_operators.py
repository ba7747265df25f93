"""The operators of an attention layer beside the KDA layer, as they are measured: the norms of the query and key heads with
the position rotation (forward, gradients), and attention over a sliding window with a few first tokens that stay visible
(forward, gradients, one token from a ring cache).

``run`` computes a case in plain torch operations in 32 bits (``own`` false) or by the library's calls
(``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.

Cases (a dict of plain values):
  op       rotary | rotary_grad | attend | attend_grad | step
  type     type of the activations: bf16, f16 or f32 (attention: bf16 or f16)
  H, Hk, d query heads, key heads, channels of a head
rotary, rotary_grad: T tokens; rot: rotated channels of a head (0: none); pairs: "halves" (i, i + rot/2) or "adjacent";
  weight: the norm has weights; fused: q and k are column ranges of one projection's rows; far: positions around a million.
attend, attend_grad: T tokens in N packed sequences of ragged lengths; W: window; S: sinks.
step: B tokens, each the next one of its own slot; W, S; full: every cache is full (else: of any length).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
THETA = 10000.0


def listed():
    return [
        # queries and keys of a decoding step of 8 tokens
        {"name": "rotary_t8_h16", "op": "rotary", "T": 8, "H": 16, "Hk": 4, "d": 128, "rot": 128, "pairs": "halves", "weight": True, "fused": True, "far": False, "type": "bf16"},
        # the same of a packed batch at full width, far into a long context
        {"name": "rotary_t65536_h32", "op": "rotary", "T": 65536, "H": 32, "Hk": 8, "d": 128, "rot": 128, "pairs": "halves", "weight": True, "fused": True, "far": True, "type": "bf16"},
        # gradients of one layer
        {"name": "rotary_grad_t8192_h16", "op": "rotary_grad", "T": 8192, "H": 16, "Hk": 16, "d": 128, "rot": 128, "pairs": "halves", "weight": True, "fused": False, "far": False, "type": "bf16"},
        # odd counts, half of the channels rotated in adjacent pairs, in 32 bits
        {"name": "rotary_grad_t5003_h5_f32", "op": "rotary_grad", "T": 5003, "H": 5, "Hk": 5, "d": 64, "rot": 32, "pairs": "adjacent", "weight": True, "fused": True, "far": False, "type": "f32"},
        # one short prompt, everything visible: latency counts
        {"name": "attend_t1024_h8", "op": "attend", "T": 1024, "N": 1, "H": 8, "Hk": 8, "d": 128, "W": 1024, "S": 0, "type": "bf16"},
        # prefill or training of a packed batch, local attention with shared key heads
        {"name": "attend_packed32768_w1024", "op": "attend", "T": 32768, "N": 24, "H": 16, "Hk": 4, "d": 128, "W": 1024, "S": 4, "type": "bf16"},
        # a long prompt, everything visible
        {"name": "attend_t8192_h16", "op": "attend", "T": 8192, "N": 1, "H": 16, "Hk": 4, "d": 128, "W": 8192, "S": 0, "type": "bf16"},
        # lengths and a window that no tile divides, narrow heads, fp16
        {"name": "attend_t5003_w333_f16", "op": "attend", "T": 5003, "N": 7, "H": 12, "Hk": 12, "d": 64, "W": 333, "S": 1, "type": "f16"},
        # gradients of one layer of local attention
        {"name": "attend_grad_t8192_w1024", "op": "attend_grad", "T": 8192, "N": 1, "H": 16, "Hk": 4, "d": 128, "W": 1024, "S": 4, "type": "bf16"},
        # gradients of ragged documents, everything visible, fp16
        {"name": "attend_grad_packed8192_f16", "op": "attend_grad", "T": 8192, "N": 5, "H": 8, "Hk": 8, "d": 64, "W": 8192, "S": 0, "type": "f16"},
        # a decoding step of two tokens, a window of 1024
        {"name": "step_b2_w1024", "op": "step", "B": 2, "H": 16, "Hk": 4, "d": 128, "W": 1024, "S": 4, "full": True, "type": "bf16"},
        # a decoding step of a full batch, caches of any length
        {"name": "step_b64_w4096", "op": "step", "B": 64, "H": 32, "Hk": 8, "d": 128, "W": 4096, "S": 4, "full": False, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_grad", "attend", "attend", "attend_grad", "step"])
    if op in ("rotary", "rotary_grad"):
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        d = rng.choice([32, 64, 128, 128, 256])
        Hk = rng.randint(1, 8)
        H = Hk * rng.choice([1, 2, 4])
        T = min(_log(rng, 1, 65000), 160_000_000 // ((H + Hk) * d * (2 if kind == "f32" else 1)))
        return {"op": op, "T": T, "H": H, "Hk": Hk, "d": d, "rot": rng.choice([0, 16, d // 2, d, d]), "pairs": rng.choice(["halves", "halves", "adjacent"]),
                "weight": rng.random() < 0.7, "fused": rng.random() < 0.5, "far": rng.random() < 0.3, "type": kind}
    kind, d = rng.choice(["bf16", "bf16", "f16"]), rng.choice([64, 128])
    Hk = rng.randint(1, 6)
    H = Hk * rng.choice([1, 2, 3, 4])
    if op == "step":
        W = _log(rng, 1, 4096)
        B = min(_log(rng, 1, 200), max(1, 64 * 4096 * 8 // (W * Hk)))
        return {"op": op, "B": B, "H": H, "Hk": Hk, "d": d, "W": W, "S": rng.choice([0, 1, 4]), "full": rng.random() < 0.5, "type": kind}
    T = _log(rng, 1, 16000)
    W = rng.choice([T, _log(rng, 1, T)])
    most = (8192 * 8192 * 16) if op == "attend" else (8192 * 1024 * 16 * 2)    # scores, the masked half of a dense square among them
    T = min(T, max(1, int(math.sqrt(most / H)) if W >= T else most // (2 * H * max(W, 128))))
    N = min(T, _log(rng, 1, 40))
    if op == "attend_grad":      # a row that sees itself alone has no gradient of its scores: they are not all like that
        T, W, N = max(T, 16), max(W, 4), min(N, max(1, T // 8))
    return {"op": op, "T": T, "N": N, "H": H, "Hk": Hk, "d": d, "W": min(W, T), "S": rng.choice([0, 0, 1, 4]), "type": kind}


def _lengths(T, N, seed):
    """N ragged lengths of one token or more that sum to T, log-uniform over a factor of 32."""
    gen = torch.Generator().manual_seed(seed)
    w = torch.exp(torch.rand(N, generator=gen, dtype=torch.float64) * math.log(32.0))
    n = 1 + torch.floor(w / w.sum() * (T - N)).to(torch.int64)
    n[0] += T - int(n.sum())
    return n


def _frequencies(rot):
    return THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    s = dict(case)
    op, H, Hk, d = case["op"], case["H"], case["Hk"], case["d"]
    if op in ("rotary", "rotary_grad"):
        T = case["T"]
        if case["fused"]:      # the rows of a projection to queries, keys and values
            wide = normal(T, (H + 2 * Hk) * d, dtype=t, std=1.5)
            s["q"], s["k"] = wide[:, :H * d].unflatten(1, (H, d)), wide[:, H * d:(H + Hk) * d].unflatten(1, (Hk, d))
        else:
            s["q"], s["k"] = normal(T, H, d, dtype=t, std=1.5), normal(T, Hk, d, dtype=t, std=1.5)
        s["w_q"], s["w_k"] = (1 + normal(d, std=0.1), 1 + normal(d, std=0.1)) if case["weight"] else (None, None)
        # packed documents: positions start again every few thousand tokens
        s["positions"] = (torch.arange(T, device="cuda") % 5000 + (1_000_000 if case["far"] else 0)).to(torch.int32)
        s["frequencies"] = _frequencies(case["rot"])
        if op == "rotary_grad":
            s["dq_out"], s["dk_out"] = normal(T, H, d, dtype=t), normal(T, Hk, d, dtype=t)
    elif op == "step":
        B, W, S = case["B"], case["W"], case["S"]
        cap = W + S
        s["q"], s["k"], s["v"] = normal(B, H, d, dtype=t), normal(B, Hk, d, dtype=t), normal(B, Hk, d, dtype=t)
        s["cache_k"], s["cache_v"] = normal(B + 1, Hk, cap, d, dtype=t), normal(B + 1, Hk, cap, d, dtype=t)
        s["slots"] = torch.randperm(B + 1, generator=gen, device="cuda")[:B].to(torch.int32)
        lo, hi = (cap, 4 * cap) if case["full"] else (0, 2 * cap)
        s["lengths"] = torch.randint(lo, hi, (B,), generator=gen, device="cuda").to(torch.int32)     # tokens before this one
        s["scale"] = d ** -0.5
    else:
        T, N = case["T"], case["N"]
        n = _lengths(T, N, seed)
        cu = torch.zeros(N + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(n, 0)
        s["cu"], s["longest"] = cu.tolist(), int(n.max())
        s["start"] = torch.repeat_interleave(cu[:-1], n).cuda()      # of every token's sequence
        # queries and keys as they come out of head norms: unit entries, a few pairs that match
        s["q"], s["k"], s["v"] = normal(T, H, d, dtype=t), normal(T, Hk, d, dtype=t), normal(T, Hk, d, dtype=t)
        s["scale"] = d ** -0.5
        if op == "attend_grad":
            s["do"] = normal(T, H, d, dtype=t)
            o, lse = _attention(s)
            s["o"], s["lse"] = o.to(t), lse
            del o
    if own:
        _plan(s, t)
    return s


def _plan(s, t):
    """The plan, workspace and output buffers that a user's program keeps."""
    import context_kda_gb300 as kda
    op = s["op"]
    like = lambda name: torch.empty(s[name].shape, dtype=t, device="cuda")
    if op in ("rotary", "rotary_grad"):
        s["phases"] = torch.from_numpy(kda.kda_rotary_phases(s["frequencies"].numpy())).cuda() if s["rot"] else None
        if op == "rotary":
            s["q_out"], s["k_out"] = like("q"), like("k")
        else:
            s["dq"], s["dk"] = like("q"), like("k")
            s["dw_q"], s["dw_k"] = (torch.empty(s["d"], device="cuda"), torch.empty(s["d"], device="cuda")) if s["weight"] else (None, None)
            s["ws"] = torch.empty(kda.kda_head_norm_rotary_workspace_bytes(s["d"]), dtype=torch.uint8, device="cuda")
    elif op == "step":
        s["out"] = like("q")
    else:
        s["plan"] = kda.kda_plan_segments(s["cu"], 1)
        s["plan_dev"] = kda.upload_plan(s["plan"])
        if op == "attend":
            s["out"], s["lse_out"] = like("q"), torch.empty(s["H"], s["T"], device="cuda")
        else:
            s["dq"], s["dk"], s["dv"] = like("q"), like("k"), like("v")
            s["o"] = s["o"].contiguous()      # as the forward call returns it
            n = kda.kda_window_attention_workspace_bytes(s["plan"], s["H"], s["Hk"], s["d"], s["W"], s["S"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


def run(s):
    return (_own if own else _plain)[s["op"]](s)


# ---- the library's calls ----------------------------------------------------------------------------


def _own_rotary(s):
    import context_kda_gb300 as kda
    kda.kda_head_norm_rotary_forward(s["q"], s["k"], True, s["w_q"], s["w_k"], EPS, s["positions"], s["phases"], s["pairs"], s["q_out"], s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_rotary_grad(s):
    import context_kda_gb300 as kda
    kda.kda_head_norm_rotary_backward(s["q"], s["k"], True, s["w_q"], s["w_k"], EPS, s["positions"], s["phases"], s["pairs"], s["dq_out"], s["dk_out"],
                                      s["dq"], s["dk"], s["dw_q"], s["dw_k"], s["ws"])
    return {"dq": s["dq"], "dk": s["dk"], "dw_q": s["dw_q"], "dw_k": s["dw_k"]}


def _own_attend(s):
    import context_kda_gb300 as kda
    kda.kda_window_attention_forward(s["plan"], s["plan_dev"], s["q"], s["k"], s["v"], s["scale"], s["W"], s["S"], s["out"], s["lse_out"])
    return {"o": s["out"], "lse": s["lse_out"]}


def _own_attend_grad(s):
    import context_kda_gb300 as kda
    kda.kda_window_attention_backward(s["plan"], s["plan_dev"], s["q"], s["k"], s["v"], s["scale"], s["W"], s["S"], s["o"], s["lse"], s["do"],
                                      s["dq"], s["dk"], s["dv"], s["ws"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _own_step(s):
    import context_kda_gb300 as kda
    kda.kda_window_attention_step(s["slots"], s["lengths"], s["q"], s["k"], s["v"], s["scale"], s["W"], s["S"], s["cache_k"], s["cache_v"], s["out"])
    return {"o": s["out"], "cache_k": s["cache_k"], "cache_v": s["cache_v"]}


# ---- the plain forms ------------------------------------------------------------------------------------


def _angles(s):
    """cos and sin [T, 1, rot / 2]; the angles of far positions take 64 bits."""
    a = s["positions"].double().unsqueeze(-1) * s["frequencies"].cuda()
    return torch.cos(a).float().unsqueeze(1), torch.sin(a).float().unsqueeze(1)


def _pairs(s, x):
    """The two channels of every rotated pair."""
    r = s["rot"]
    return (x[..., :r // 2], x[..., r // 2:r]) if s["pairs"] == "halves" else (x[..., 0:r:2], x[..., 1:r:2])


def _rotate(s, x, c, n):
    if not s["rot"]:
        return x
    a, b = _pairs(s, x)
    out = x.clone()
    p, q = _pairs(s, out)
    p.copy_(a * c - b * n)
    q.copy_(a * n + b * c)
    return out


def _plain_rotary(s):
    c, n = _angles(s)

    def one(x, w):
        v = x.float()
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
        return _rotate(s, v if w is None else v * w, c, n).to(x.dtype)

    return {"q": one(s["q"], s["w_q"]), "k": one(s["k"], s["w_k"])}


def _plain_rotary_grad(s):
    c, n = _angles(s)

    def one(x, w, g):
        v, g = x.float(), _rotate(s, g.float(), c, -n)
        inv = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
        hat = v * inv
        dw = None if w is None else (g * hat).sum((0, 1))
        e = g if w is None else g * w
        return (inv * (e - hat * (e * hat).mean(-1, keepdim=True))).to(x.dtype), dw

    (dq, dw_q), (dk, dw_k) = one(s["q"], s["w_q"], s["dq_out"]), one(s["k"], s["w_k"], s["dk_out"])
    return {"dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}


def _blocks(s):
    """Rows in blocks of n, each against its own and the block before, which hold every window: n, blocks, and the rows' and
    keys' tokens with what is visible."""
    T, W = s["T"], min(s["W"], s["longest"])
    n = min(T, max(W, 128))
    count = -(-T // n)
    width = 2 * n if count > 1 else n
    i = torch.arange(count * n, device="cuda").view(count, n, 1)
    j = torch.arange(count, device="cuda").view(count, 1, 1) * n + torch.arange(width, device="cuda") - (width - n)
    start = torch.nn.functional.pad(s["start"], (0, count * n - T), value=T).view(count, n, 1)
    return n, count, width, (j <= i) & (i - j < W) & (j >= start)


def _rows(x, n, count):
    """[T, heads, d] in fp32 as [blocks, heads, n, d], zeros behind the last token."""
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, n * count - x.shape[0]))
    return x.view(count, n, *x.shape[1:]).transpose(1, 2)


def _keys(x, n, count, width):
    """The same for keys: every block's own rows behind those of the block before."""
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, width - n, n * count - x.shape[0]))
    return x.unfold(0, width, n).permute(0, 1, 3, 2)


def _sinks(s):
    """Every token's sinks behind its window: their tokens [T, S] and whether they are visible."""
    at = s["start"].view(-1, 1) + torch.arange(s["S"], device="cuda")
    return at.clamp(max=s["T"] - 1), at <= torch.arange(s["T"], device="cuda").view(-1, 1) - s["W"]


def _probabilities(s, lse=None):
    """exp(score - lse) of the window [blocks, Hk, g n, width] and of the sinks [T, Hk, g, S], with lse [H, T] (computed where it is not given)."""
    T, H, Hk, d = s["T"], s["H"], s["Hk"], s["d"]
    g = H // Hk
    n, count, width, seen = _blocks(s)
    q = _rows(s["q"] * 1, n, count).reshape(count, Hk, g * n, d)
    p = torch.matmul(q, _keys(s["k"], n, count, width).transpose(-1, -2)).mul_(s["scale"])
    p.view(count, Hk, g, n, width).masked_fill_(~seen.view(count, 1, 1, n, width), float("-inf"))
    at, open_ = _sinks(s)
    ps = torch.matmul(s["q"].float().view(T, Hk, g, d), s["k"].float()[at].permute(0, 2, 3, 1)) * s["scale"]      # [T, Hk, g, S]
    ps = ps.masked_fill(~open_.view(T, 1, 1, -1), float("-inf"))
    by_row = lambda x: x.reshape(count, Hk, g, n).permute(0, 3, 1, 2).reshape(count * n, Hk, g)[:T]      # to [T, Hk, g]
    to_row = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * count - T)).view(count, n, Hk, g).permute(0, 2, 3, 1).reshape(count, Hk, g * n, 1)
    if lse is None:
        top = by_row(p.amax(-1))
        if s["S"]:
            top = torch.maximum(top, ps.amax(-1))
        p.sub_(to_row(top)).exp_()
        ps = torch.exp(ps - top.unsqueeze(-1))
        total = by_row(p.sum(-1)) + ps.sum(-1)
        p.div_(to_row(total).clamp(min=1e-30))
        lse = (top + torch.log(total)).reshape(T, H).t().contiguous()
        return p, ps / total.unsqueeze(-1), lse
    lse = lse.t().reshape(T, Hk, g)
    return p.sub_(to_row(lse)).exp_(), torch.exp(ps - lse.unsqueeze(-1)), None


def _attention(s):
    T, H, Hk, d = s["T"], s["H"], s["Hk"], s["d"]
    n, count, width, _ = _blocks(s)
    p, ps, lse = _probabilities(s)
    o = torch.matmul(p, _keys(s["v"], n, count, width)).view(count, H, n, d).transpose(1, 2).reshape(-1, H, d)[:T]
    at, _ = _sinks(s)
    return o + torch.matmul(ps, s["v"].float()[at].transpose(1, 2)).view(T, H, d), lse


def _plain_attend(s):
    o, lse = _attention(s)
    return {"o": o.to(s["q"].dtype), "lse": lse}


def _fold(x, n, count, width, T):
    """The gradients of _keys' blocks [blocks, Hk, width, d] back to tokens [T, Hk, d]."""
    x = x.transpose(1, 2)
    out = x[:, width - n:].clone()
    if width > n:
        out[:-1] += x[1:, :n]
    return out.reshape(count * n, *x.shape[2:])[:T]


def _plain_attend_grad(s):
    T, H, Hk, d = s["T"], s["H"], s["Hk"], s["d"]
    g, kind = H // Hk, s["q"].dtype
    n, count, width, _ = _blocks(s)
    p, ps, _ = _probabilities(s, s["lse"])
    k, v = _keys(s["k"], n, count, width), _keys(s["v"], n, count, width)
    q, do = (_rows(s[x], n, count).reshape(count, Hk, g * n, d) for x in ("q", "do"))
    at, _ = _sinks(s)
    ks, vs = s["k"].float()[at].transpose(1, 2), s["v"].float()[at].transpose(1, 2)     # [T, Hk, S, d]
    q1, do1 = s["q"].float().view(T, Hk, g, d), s["do"].float().view(T, Hk, g, d)
    # p (dp - sum p dp)
    ds, dss = torch.matmul(do, v.transpose(-1, -2)).mul_(p), torch.matmul(do1, vs.transpose(-1, -2)) * ps
    mean = ds.sum(-1, keepdim=True)
    mean1 = mean.view(count, Hk, g, n).permute(0, 3, 1, 2).reshape(count * n, Hk, g, 1)[:T] + dss.sum(-1, keepdim=True)
    mean = torch.nn.functional.pad(mean1.squeeze(-1), (0, 0, 0, 0, 0, n * count - T)).view(count, n, Hk, g).permute(0, 2, 3, 1).reshape(count, Hk, g * n, 1)
    ds.addcmul_(p, mean, value=-1)
    dss = dss - ps * mean1
    dv = _fold(torch.matmul(p.transpose(-1, -2), do), n, count, width, T)
    dk = _fold(torch.matmul(ds.transpose(-1, -2), q), n, count, width, T)
    dq = torch.matmul(ds, k).view(count, H, n, d).transpose(1, 2).reshape(-1, H, d)[:T] + torch.matmul(dss, ks).view(T, H, d)
    if s["S"]:      # every sequence's sinks collect from all its rows: a product with the rows' sequences
        starts, seq = torch.unique(s["start"], return_inverse=True)
        member = torch.nn.functional.one_hot(seq, len(starts)).float().t()
        at1 = starts.view(-1, 1) + torch.arange(s["S"], device="cuda")
        real = at1 <= torch.cat([starts[1:], starts.new_tensor([T])]).view(-1, 1) - 1
        for into, part in ((dv, torch.matmul(ps.transpose(-1, -2), do1)), (dk, torch.matmul(dss.transpose(-1, -2), q1))):
            total = torch.matmul(member, part.transpose(1, 2).reshape(T, -1)).view(len(starts), s["S"], Hk, d)
            into[at1[real]] += total[real]
    return {"dq": (dq * s["scale"]).to(kind), "dk": (dk * s["scale"]).to(kind), "dv": dv.to(kind)}


def _plain_step(s):
    B, H, Hk, d, W, S = (s[x] for x in ("B", "H", "Hk", "d", "W", "S"))
    slots, n = s["slots"].long(), s["lengths"].long()
    row = torch.where(n < S, n, S + (n - S) % W)
    s["cache_k"][slots, :, row], s["cache_v"][slots, :, row] = s["k"], s["v"]
    k, v = s["cache_k"][slots].float(), s["cache_v"][slots].float()
    x = torch.matmul(s["q"].float().view(B, Hk, H // Hk, d), k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill(torch.arange(W + S, device="cuda") > n.view(B, 1, 1, 1), float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    return {"o": o.view(B, H, d).to(s["q"].dtype), "cache_k": s["cache_k"], "cache_v": s["cache_v"]}


_own = {"rotary": _own_rotary, "rotary_grad": _own_rotary_grad, "attend": _own_attend, "attend_grad": _own_attend_grad, "step": _own_step}
_plain = {"rotary": _plain_rotary, "rotary_grad": _plain_rotary_grad, "attend": _plain_attend, "attend_grad": _plain_attend_grad,
          "step": _plain_step}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------


def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))


def _exact_turn(s):
    """The rotation of every token as a complex number for each pair."""
    return torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(s["positions"].double(), s["frequencies"].cuda())).unsqueeze(1)


def _exact_turned(s, x, turn):
    r, out = s["rot"], x.clone()
    if r and s["pairs"] == "adjacent":
        out[..., :r] = torch.view_as_real(torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn).flatten(-2)
    elif r:
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
        out[..., :r] = torch.cat([z.real, z.imag], -1)
    return out


def _exact_rotary(s):
    turn, out = _exact_turn(s), {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w_" + n]
        x = x * (x.square().sum(-1, keepdim=True) / s["d"] + EPS).rsqrt()
        out[n] = _exact_turned(s, x if w is None else x * w.double(), turn)
    return out


def _exact_rotary_grad(s):
    turn, out = _exact_turn(s).conj(), {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w_" + n]
        g = _exact_turned(s, s["d%s_out" % n].double(), turn)
        size = (x.square().sum(-1, keepdim=True) / s["d"] + EPS).sqrt()
        out["dw_" + n] = None if w is None else torch.einsum("thd,thd->d", g, x / size)
        g = g if w is None else g * w.double()
        out["d" + n] = g / size - x * (g * x).sum(-1, keepdim=True) / (s["d"] * size ** 3)
    return {x: out[x] for x in ("dq", "dk", "dw_q", "dw_k")}


def _exact_parts(s):
    """Pieces of a sequence's rows for one key head: the rows, the keys that any of them sees, and which sees which."""
    for a, b in zip(s["cu"][:-1], s["cu"][1:]):
        for lo in range(a, b, 1024):
            hi = min(b, lo + 1024)
            first = max(a, lo - s["W"] + 1)
            j = torch.cat([torch.arange(a, min(first, a + s["S"])), torch.arange(first, hi)]).cuda()
            i = torch.arange(lo, hi, device="cuda").view(-1, 1)
            seen = (j <= i) & ((i - j < s["W"]) | (j - a < s["S"]))
            for h in range(s["Hk"]):
                yield lo, hi, j, seen, h


def _exact_scores(s, lo, hi, j, seen, h):
    g = s["H"] // s["Hk"]
    q, k = s["q"][lo:hi, h * g:(h + 1) * g].double(), s["k"][j, h].double()
    x = s["scale"] * torch.einsum("ihd,jd->hij", q, k)
    return x.masked_fill(~seen, -math.inf), q, k


def _exact_attend(s):
    g = s["H"] // s["Hk"]
    o, lse = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), torch.empty(s["H"], s["T"], dtype=torch.float64, device="cuda")
    for lo, hi, j, seen, h in _exact_parts(s):
        x, _, _ = _exact_scores(s, lo, hi, j, seen, h)
        l = torch.logsumexp(x, -1)
        lse[h * g:(h + 1) * g, lo:hi] = l
        o[lo:hi, h * g:(h + 1) * g] = torch.einsum("hij,jd->ihd", torch.exp(x - l.unsqueeze(-1)), s["v"][j, h].double())
    return {"o": o, "lse": lse}


def _exact_attend_grad(s):
    g = s["H"] // s["Hk"]
    dq, dk, dv = (torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in ("q", "k", "v"))
    for lo, hi, j, seen, h in _exact_parts(s):
        x, q, k = _exact_scores(s, lo, hi, j, seen, h)
        p = torch.softmax(x, -1)
        do = s["do"][lo:hi, h * g:(h + 1) * g].double()
        dv[j, h] += torch.einsum("hij,ihd->jd", p, do)
        dp = torch.einsum("ihd,jd->hij", do, s["v"][j, h].double())
        ds = s["scale"] * p * (dp - (p * dp).sum(-1, keepdim=True))
        dq[lo:hi, h * g:(h + 1) * g] = torch.einsum("hij,jd->ihd", ds, k)
        dk[j, h] += torch.einsum("hij,ihd->jd", ds, q)
    return {"dq": dq, "dk": dk, "dv": dv}


def _exact_step(s):
    g, S, W = s["H"] // s["Hk"], s["S"], s["W"]
    ck, cv = s["cache_k"].double(), s["cache_v"].double()
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (slot, n) in enumerate(zip(s["slots"].tolist(), s["lengths"].tolist())):
        row = n if n < S else S + (n - S) % W
        ck[slot, :, row], cv[slot, :, row] = s["k"][b].double(), s["v"][b].double()
        rows = min(n + 1, S + W)
        x = s["scale"] * torch.einsum("hgd,hjd->hgj", s["q"][b].double().view(s["Hk"], g, -1), ck[slot, :, :rows])
        o[b] = torch.einsum("hgj,hjd->hgd", torch.softmax(x, -1), cv[slot, :, :rows]).reshape(s["H"], -1)
    return {"o": o, "cache_k": ck, "cache_v": cv}


_exact = {"rotary": _exact_rotary, "rotary_grad": _exact_rotary_grad, "attend": _exact_attend, "attend_grad": _exact_attend_grad,
          "step": _exact_step}


def _visible(case):
    """Pairs of a query and a key that it sees, of one head; lengths as drawn for one seed."""
    W, S, total = case["W"], case["S"], 0
    for n in _lengths(case["T"], case["N"], 0).tolist():
        m = min(n, W)
        total += m * (m + 1) // 2 + (n - m) * W                          # of the window
        k = max(0, n - W)                                                # rows that a sink has left the window of
        total += sum(max(0, k - a) for a in range(min(S, n)))
    return total


def work(case):
    """Bytes: every input once, every output once.  Operations: an exponential counts as one."""
    op, e, H, Hk, d = case["op"], BYTES[case["type"]], case["H"], case["Hk"], case["d"]
    if op in ("rotary", "rotary_grad"):
        n = case["T"] * (H + Hk) * d
        weights = 2 * d * 4 if case["weight"] else 0
        if op == "rotary":
            return {"bytes": n * 2 * e + case["T"] * 4 + weights, "flops": n * 8}
        return {"bytes": n * 3 * e + case["T"] * 4 + 2 * weights, "flops": n * 16}
    if op == "step":
        B, cap = case["B"], case["W"] + case["S"]
        rows = B * (cap if case["full"] else 0.75 * cap)                 # half of the lengths fill the cache, the others half of it
        return {"bytes": 2 * rows * Hk * d * e + B * (2 * H + 4 * Hk) * d * e, "flops": rows * H * (4 * d + 4)}
    n, pairs = case["T"] * d * e, _visible(case) * H
    if op == "attend":
        return {"bytes": n * 2 * (H + Hk) + case["T"] * H * 4, "flops": pairs * (4 * d + 4)}
    return {"bytes": n * (4 * H + 4 * Hk) + case["T"] * H * 4, "flops": pairs * (10 * d + 6)}
