"""What is measured of the state-space layer and the gradient clipping.

Three families, in the library's layouts (heads first, tokens next, channels
innermost):

conv    the short causal depthwise convolution over tokens that precedes a
        recurrent layer: y_t = act(bias + sum_j w_j x_{t-(W-1)+j}), for prompts,
        for training (with its gradients) and for single tokens.
scan    the selective state-space scan
            S_t = exp(dt_t A) S_{t-1} + dt_t v_t k_t^T,   y_t = S_t q_t + D v_t
        (v is the layer's x, k its B, q its C; q and k are shared by the H / G
        heads of a group), for prompts, for training and for single tokens.
clip    the global 2-norm of many gradient tensors and their clipping by it.

`own` false: the plain form, in elementary torch operations in 32 bits (sums of
logarithms in 64). `own` true: the framework's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens per block of the plain form's matrix products


# ------------------------------------------------------------------ cases
def _conv(op, **k):
    return dict(op=op, act="bf16", B=1, H=1, T=1, d=64, W=4, bias=True, silu=True, state=False, ragged=False) | k


def _scan(op, **k):
    return dict(op=op, act="bf16", B=1, H=1, G=1, T=1, P=64, N=128, D=True, state=False, ragged=False) | k


def listed():
    return [
        # a training step of the convolution in front of the 1.3B layer (4 x 8 heads of 256, 2K tokens)
        _conv("conv_train", name="conv train 4x8x2048x256", B=4, H=8, T=2048, d=256),
        # a padded batch of prompts that continue earlier ones, full precision, odd sizes
        _conv("conv_prompt", name="conv prompt f32 ragged", act="f32", B=3, H=5, T=1021, d=72, W=3, silu=False,
              state=True, ragged=True),
        # one new token for each of 64 sequences
        _conv("conv_step", name="conv step 64 rows", B=64, H=32, d=64),
        # the shortest prompts, where the call itself counts
        _scan("scan_prompt", name="scan prompt 37 tokens", B=1, H=8, T=37, N=64),
        # ordinary prompts, a batch of them
        _scan("scan_prompt", name="scan prompt 4x32x2048", B=4, H=32, T=2048),
        # one long prompt: few rows, a long axis
        _scan("scan_prompt", name="scan prompt 1x32x16384", B=1, H=32, T=16384),
        # a training step, all heads on one q and k
        _scan("scan_train", name="scan train 2x64x2048", B=2, H=64, T=2048),
        # full precision, grouped heads, odd sizes, a padded batch that starts from states
        _scan("scan_train", name="scan train f32 ragged", act="f32", B=2, H=6, G=2, T=509, P=48, N=40, state=True,
              ragged=True),
        # single tokens: one sequence, and a serving batch
        _scan("scan_step", name="scan step 1 row", B=1, H=32, N=64),
        _scan("scan_step", name="scan step 64 rows", B=64, H=32),
        # the gradients of a large model's layer: a few large matrices and many small vectors
        dict(op="clip", name="clip 64M values", act="mixed", big=12, big_n=5_242_880, small=24, small_n=1031),
        # many small tensors, where the calls count
        dict(op="clip", name="clip 160 small", act="mixed", big=10, big_n=16_384, small=150, small_n=517),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_train", "conv_prompt", "conv_step", "scan_prompt", "scan_prompt", "scan_train", "scan_train",
                     "scan_step", "clip"])
    act = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "clip":
        big = _log(rng, 1, 24)
        return dict(op=op, act=rng.choice(["mixed", "bf16", "f32"]), big=big, big_n=_log(rng, 1000, 60_000_000 // big),
                    small=rng.randint(0, 200), small_n=_log(rng, 1, 4000))
    if op.startswith("conv"):
        d = rng.choice([8, 24, 33, 64, 64, 72, 128, 128, 200, 256])
        if op == "conv_step":
            B, H, T = _log(rng, 1, 128), _log(rng, 1, 32), 1
        else:
            T = _log(rng, 1, 8192)
            H = min(_log(rng, 1, 32), max(1, 16_000_000 // (T * d)))
            B = min(_log(rng, 1, 8), max(1, 16_000_000 // (T * d * H)))
        return _conv(op, act=act, B=B, H=H, T=T, d=d, W=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.7,
                     silu=rng.random() < 0.7, state=rng.random() < 0.4, ragged=T > 1 and rng.random() < 0.4)
    P, N = rng.choice([32, 48, 64, 64, 64, 96, 128]), rng.choice([16, 40, 64, 64, 128, 128, 128])
    G = rng.choice([1, 1, 1, 2, 4])
    if op == "scan_step":
        B, H, T = _log(rng, 1, 64), G * _log(rng, 1, 32 // G), 1
    else:
        most = (260_000 if op == "scan_train" else 500_000) * 8192 // max(8192, P * N)
        most = most // 8 if act == "f32" else most
        T = _log(rng, 1, 16_384)
        H = G * min(_log(rng, 1, 64 // G), max(1, most // (T * G)))
        B = min(_log(rng, 1, 8), max(1, most // (T * H)))
    return _scan(op, act=act, B=B, H=H, G=G, T=T, P=P, N=N, D=rng.random() < 0.7, state=rng.random() < 0.4,
                 ragged=T > 1 and rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=DEV) * (hi - lo) + lo

    st = {"case": c}
    if c["op"] == "clip":
        sizes = [c["big_n"]] * c["big"] + [c["small_n"]] * c["small"]
        kinds = {"bf16": [torch.bfloat16], "f32": [torch.float32], "mixed": [torch.bfloat16, torch.float32]}[c["act"]]
        st["grads"] = [normal(n, dtype=kinds[i % len(kinds)], scale=0.02) for i, n in enumerate(sizes)]
        # the clipped gradients go to one flat buffer of each type, as gradient buckets are laid out
        st["flat"], st["out"] = _buckets(st["grads"], lambda x: x.dtype)
        st["max_norm"] = 1.0
        return st
    a, B, H, T = ACT[c["act"]], c["B"], c["H"], c["T"]
    # a padded batch has one full row; the others end anywhere, the start included
    st["lengths"] = None
    if c["ragged"]:
        st["lengths"] = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        st["lengths"][0] = T
    if c["op"].startswith("conv"):
        d, W = c["d"], c["W"]
        st["x"] = normal(B, H, T, d, dtype=a)
        st["w"] = normal(H, d, W, scale=W ** -0.5)
        st["bias"] = normal(H, d, scale=0.1) if c["bias"] else None
        step = c["op"] == "conv_step"
        st["state"] = normal(B, H, W - 1, d, dtype=a) if c["state"] or step else None
        if step:
            st["x"] = st["x"].reshape(B, H, d)
            st["y"] = torch.empty_like(st["x"])
        if c["op"] == "conv_train":
            st["dy"] = normal(B, H, T, d, dtype=a)
        return st
    G, P, N = c["G"], c["P"], c["N"]
    st["q"], st["k"] = normal(B, G, T, N, dtype=a), normal(B, G, T, N, dtype=a)
    st["v"] = normal(B, H, T, P, dtype=a)
    st["dt"] = torch.exp(uniform(math.log(1e-3), math.log(1e-1), B, H, T))
    st["A"] = -uniform(1.0, 16.0, H)
    st["D"] = normal(H) if c["D"] else None
    step = c["op"] == "scan_step"
    st["S"] = normal(B, H, P, N, scale=0.3) if c["state"] or step else None
    if step:
        for n in ("q", "k", "v", "dt"):
            st[n] = st[n].squeeze(2)
        st["y"] = torch.empty_like(st["v"])
    if c["op"] == "scan_train":
        st["dy"] = normal(B, H, T, P, dtype=a)
    return st


def _buckets(tensors, held_as):
    """A flat buffer for each type among `tensors`, each tensor's place on a multiple of 8 values, and the places."""
    flat, places = [], [None] * len(tensors)
    for kind in sorted({x.dtype for x in tensors}, key=str):
        of_kind = [i for i, x in enumerate(tensors) if x.dtype == kind]
        sizes = [(tensors[i].numel() + 7) // 8 * 8 for i in of_kind]
        flat.append(torch.zeros(sum(sizes), dtype=held_as(tensors[of_kind[0]]), device=DEV))
        for i, part in zip(of_kind, flat[-1].split(sizes)):
            places[i] = part[:tensors[i].numel()]
    return flat, places


# ------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import test_weight_layers_chunk_b200 as E
    c = s["case"]
    op = c["op"]
    if op == "clip":
        norm = E.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
        return {"norm": norm, "out": s["flat"]}
    if op == "conv_step":
        y = E.short_conv_step(s["x"], s["state"], s["w"], s["bias"], silu=c["silu"], out=s["y"])
        return {"y": y, "state": s["state"]}
    if op == "conv_prompt":
        y, end = E.short_conv_fwd(s["x"], s["w"], s["bias"], s["state"], s["lengths"], silu=c["silu"], return_state=True)
        return {"y": y, "state": end}
    if op == "conv_train":
        y, _ = E.short_conv_fwd(s["x"], s["w"], s["bias"], s["state"], s["lengths"], silu=c["silu"])
        g = E.short_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], s["state"], lengths=s["lengths"], silu=c["silu"])
        return {"y": y, "dx": g["dx"], "dw": g["dw"], "dbias": g["dbias"], "dstate": g["dstate"]}
    if op == "scan_step":
        y = E.ssm_step(s["q"], s["k"], s["v"], s["dt"], s["S"], s["A"], s["D"], out=s["y"])
        return {"y": y, "S": s["S"]}
    if op == "scan_prompt":
        y, S_end, _ = E.ssm_scan_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["D"], s["S"], s["lengths"])
        return {"y": y, "S": S_end}
    y, S_end, saved = E.ssm_scan_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["D"], s["S"], s["lengths"],
                                     save_states=True)
    g = E.ssm_scan_bwd(s["q"], s["k"], s["v"], s["dt"], s["A"], saved, s["dy"], s["D"], lengths=s["lengths"])
    return {"y": y, "S": S_end, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "ddt": g["ddt"], "dA": g["dA"],
            "dD": g["dD"], "dS0": g["dS0"] if s["S"] is not None else None}


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "clip":
        norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
        scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        [o.copy_(x.float() * scale) for o, x in zip(s["out"], s["grads"])]
        return {"norm": norm, "out": s["flat"]}
    a = ACT[c["act"]]
    if op == "conv_step":
        seq = torch.cat([s["state"].float(), s["x"].float().unsqueeze(2)], dim=2)
        z = torch.einsum("bhtd,hdt->bhd", seq, s["w"])
        z = z if s["bias"] is None else z + s["bias"]
        s["state"].copy_(seq[:, :, 1:])
        return {"y": (z / (1 + torch.exp(-z)) if c["silu"] else z).to(a), "state": s["state"]}
    if op == "conv_prompt":
        y, end = _conv_forward(s["x"].float(), s["w"], s["bias"], None if s["state"] is None else s["state"].float(),
                               s["lengths"], c["silu"])
        return {"y": y.to(a), "state": end.to(a)}
    if op == "conv_train":
        leaf = {n: s[n].float().requires_grad_() for n in ("x", "w", "bias", "state") if s[n] is not None}
        y, _ = _conv_forward(leaf["x"], leaf["w"], leaf.get("bias"), leaf.get("state"), s["lengths"], c["silu"])
        g = dict(zip(leaf, torch.autograd.grad(y, list(leaf.values()), s["dy"].float())))
        return {"y": y.detach().to(a), "dx": g["x"].to(a), "dw": g["w"], "dbias": g.get("bias"),
                "dstate": g["state"].to(a) if "state" in g else None}
    if op == "scan_step":
        per = c["H"] // c["G"]
        q, k = (s[n].float().repeat_interleave(per, 1) for n in ("q", "k"))
        v, dt = s["v"].float(), s["dt"]
        S = s["S"] * torch.exp(dt * s["A"])[..., None, None] + (dt[..., None] * v)[..., None] * k[:, :, None]
        y = (S * q[:, :, None]).sum(-1)
        y = y if s["D"] is None else y + s["D"][:, None] * v
        s["S"].copy_(S)
        return {"y": y.to(a), "S": s["S"]}
    names = ("q", "k", "v", "dt", "A", "D", "S")
    if op == "scan_prompt":
        y, S_end = _scan_forward(*(None if s[n] is None else s[n].float() for n in names), s["lengths"])
        return {"y": y.to(a), "S": S_end}
    leaf = {n: s[n].float().requires_grad_() for n in names if s[n] is not None}
    y, S_end = _scan_forward(*(leaf.get(n) for n in names), s["lengths"])
    g = dict(zip(leaf, torch.autograd.grad(y, list(leaf.values()), s["dy"].float())))
    return {"y": y.detach().to(a), "S": S_end.detach(), "dq": g["q"].to(a), "dk": g["k"].to(a), "dv": g["v"].to(a),
            "ddt": g["dt"], "dA": g["A"], "dD": g.get("D"), "dS0": g.get("S")}


def _valid(lengths, B, T):
    """[B, 1, T]: which tokens a padded batch has."""
    at = torch.arange(T, device=DEV)
    return torch.ones(B, 1, T, dtype=torch.bool, device=DEV) if lengths is None else at < lengths[:, None, None]


def _conv_forward(x, w, bias, state, lengths, silu):
    B, H, T, d = x.shape
    W = w.shape[-1]
    there = _valid(lengths, B, T)[..., None]
    x = torch.where(there, x, 0.0)
    head = torch.zeros(B, H, W - 1, d, device=DEV) if state is None else state
    seq = torch.cat([head, x], dim=2)
    z = torch.einsum("bhtdw,hdw->bhtd", seq.unfold(2, W, 1), w)
    z = z if bias is None else z + bias[:, None]
    y = torch.where(there, z / (1 + torch.exp(-z)) if silu else z, 0.0)
    first = torch.full((B,), T, device=DEV) if lengths is None else lengths.long()
    at = first[:, None] + torch.arange(W - 1, device=DEV)
    end = torch.gather(seq, 2, at[:, None, :, None].expand(B, H, W - 1, d))
    return y, end


def _scan_forward(q, k, v, dt, A, D, S0, lengths):
    """The scan over blocks of CHUNK tokens as matrix products; the blocks'
    states meet through the matrix of decays between blocks."""
    B, G, T, N = q.shape
    H, P = v.shape[1], v.shape[-1]
    there = _valid(lengths, B, T)
    x, step = torch.where(there[..., None], v, 0.0), torch.where(there, dt, 0.0)
    q, k = torch.where(there[..., None], q, 0.0), torch.where(there[..., None], k, 0.0)
    Q = min(CHUNK, T)
    C = -(-T // Q)
    pad = C * Q - T
    x_, q_, k_ = (torch.nn.functional.pad(t, (0, 0, 0, pad)) for t in (x, q, k))
    step_ = torch.nn.functional.pad(step, (0, pad))
    xc = x_.view(B, H, C, Q, P) * step_.view(B, H, C, Q, 1)
    qc, kc = q_.view(B, G, 1, C, Q, N), k_.view(B, G, 1, C, Q, N)
    log = (step_.double() * A.double()[:, None]).view(B, H, C, Q)
    cum = log.cumsum(-1)
    lower = torch.ones(Q, Q, dtype=torch.bool, device=DEV).tril()
    decay = (cum[..., :, None] - cum[..., None, :]).masked_fill(~lower, -math.inf).exp().float()
    score = (qc @ kc.transpose(-1, -2)).expand(B, G, H // G, C, Q, Q).reshape(B, H, C, Q, Q)
    y = (score * decay) @ xc
    # each block's own state, then the states at the blocks' starts and the end
    left = (cum[..., -1:] - cum).exp().float()
    kh = kc.expand(B, G, H // G, C, Q, N).reshape(B, H, C, Q, N)
    mine = (xc * left[..., None]).transpose(-1, -2) @ kh
    start = torch.zeros(B, H, 1, P, N, device=DEV) if S0 is None else S0[:, :, None]
    mine = torch.cat([start, mine], dim=2).view(B, H, C + 1, P * N)
    total = torch.nn.functional.pad(cum[..., -1], (1, 0)).cumsum(-1)
    below = torch.ones(C + 1, C + 1, dtype=torch.bool, device=DEV).tril()
    between = (total[..., :, None] - total[..., None, :]).masked_fill(~below, -math.inf).exp().float()
    states = (between @ mine).view(B, H, C + 1, P, N)
    qh = qc.expand(B, G, H // G, C, Q, N).reshape(B, H, C, Q, N)
    y = y + (qh * cum.exp().float()[..., None]) @ states[:, :, :-1].transpose(-1, -2)
    y = y.view(B, H, C * Q, P)[:, :, :T]
    y = y if D is None else y + D[:, None, None] * x
    return torch.where(there[..., None], y, 0.0), states[:, :, -1]


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """From the definitions, token by token, in 64 bits."""
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "clip":
        wide = [x.double() for x in s["grads"]]
        norm = math.sqrt(sum(float((x * x).sum()) for x in wide))
        scale = min(1.0, s["max_norm"] / (norm + 1e-6))
        flat, out = _buckets(s["grads"], lambda x: torch.float64)
        for o, x in zip(out, wide):
            o.copy_(x * scale)
        return {"norm": torch.tensor(norm, dtype=torch.float64), "out": flat}
    s = {n: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for n, v in s.items()}
    B, H, T = c["B"], c["H"], c["T"]
    ends = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    if op.startswith("conv"):
        return _exact_conv(s, c, B, H, T, ends)
    return _exact_scan(s, c, B, H, T, ends)


def _exact_conv(s, c, B, H, T, ends):
    d, W = c["d"], c["W"]
    x = s["x"].reshape(B, H, T, d)
    there = (torch.arange(T, device=DEV) < ends[:, None])[:, None, :, None].expand(B, H, T, d)
    seq = torch.zeros(B, H, W - 1 + T, d, dtype=torch.float64, device=DEV)
    if s["state"] is not None:
        seq[:, :, :W - 1] = s["state"]
    seq[:, :, W - 1:][there] = x[there]
    z = torch.zeros_like(x)
    for j in range(W):
        z += s["w"][:, None, :, j] * seq[:, :, j:j + T]
    if s["bias"] is not None:
        z += s["bias"][:, None]
    sig = torch.sigmoid(z)
    y = (z * sig if c["silu"] else z) * there
    end = torch.stack([seq[b, :, int(e):int(e) + W - 1] for b, e in enumerate(ends)])
    if c["op"] == "conv_step":
        return {"y": y[:, :, 0], "state": end}
    if c["op"] == "conv_prompt":
        return {"y": y, "state": end}
    dz = s["dy"] * there
    if c["silu"]:
        dz = dz * (sig + z * sig * (1 - sig))
    dseq, dw = torch.zeros_like(seq), torch.zeros_like(s["w"])
    for j in range(W):
        dseq[:, :, j:j + T] += s["w"][:, None, :, j] * dz
        dw[:, :, j] = (dz * seq[:, :, j:j + T]).sum((0, 2))
    return {"y": y, "dx": dseq[:, :, W - 1:] * there, "dw": dw,
            "dbias": None if s["bias"] is None else dz.sum((0, 2)),
            "dstate": None if s["state"] is None else dseq[:, :, :W - 1]}


def _exact_scan(s, c, B, H, T, ends):
    G, P, N = c["G"], c["P"], c["N"]
    per = H // G
    q, k = s["q"].reshape(B, G, T, N), s["k"].reshape(B, G, T, N)
    v, dt, A = s["v"].reshape(B, H, T, P), s["dt"].reshape(B, H, T), s["A"]
    S = torch.zeros(B, H, P, N, dtype=torch.float64, device=DEV) if s["S"] is None else s["S"].clone()
    there = torch.arange(T, device=DEV) < ends[:, None]
    dt = dt * there[:, None]
    y = torch.zeros_like(v)

    def heads(x, t):
        return x[:, :, t].repeat_interleave(per, 1)

    def forward(S, t):
        S = S * torch.exp(dt[:, :, t] * A)[..., None, None]
        return S.add_((dt[:, :, t, None] * v[:, :, t])[..., None] * heads(k, t)[:, :, None])

    marks, step = [], 64
    for t in range(T):
        if t % step == 0:
            marks.append(S)
        S = forward(S, t)
        y[:, :, t] = (S @ heads(q, t)[..., None])[..., 0]
    if s["D"] is not None:
        y += s["D"][:, None, None] * v
    y *= there[:, None, :, None]
    if c["op"] != "scan_train":
        return {"y": y[:, :, 0] if c["op"] == "scan_step" else y, "S": S}
    dy = s["dy"] * there[:, None, :, None]
    dS = torch.zeros_like(S)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    ddt, dA = torch.zeros_like(dt), torch.zeros_like(A)
    for m in reversed(range(len(marks))):
        path = [marks[m]]
        for t in range(m * step, min(T, m * step + step)):
            path.append(forward(path[-1], t))
        for t in reversed(range(m * step, min(T, m * step + step))):
            before, now = path[t - m * step], path[t - m * step + 1]
            dS = dS + dy[:, :, t, :, None] * heads(q, t)[:, :, None]
            dq[:, :, t] = (dy[:, :, t, None] @ now)[:, :, 0].view(B, G, per, N).sum(2)
            du = (dS @ heads(k, t)[..., None])[..., 0]
            dv[:, :, t] = dt[:, :, t, None] * du
            dk[:, :, t] = ((dt[:, :, t, None] * v[:, :, t])[:, :, None] @ dS)[:, :, 0].view(B, G, per, N).sum(2)
            dS = dS * torch.exp(dt[:, :, t] * A)[..., None, None]
            dlog = (dS * before).sum((-1, -2))
            ddt[:, :, t] = (du * v[:, :, t]).sum(-1) + A * dlog
            dA += (dt[:, :, t] * dlog).sum(0)
        del path
    mask = there[:, None, :]
    dv, dD = dv * mask[..., None], None
    if s["D"] is not None:
        dv += s["D"][:, None, None] * dy
        dD = (dy * v).sum((0, 2, 3))
    return {"y": y, "S": S, "dq": dq * mask[..., None], "dk": dk * mask[..., None], "dv": dv, "ddt": ddt * mask,
            "dA": dA, "dD": dD, "dS0": None if s["S"] is None else dS}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = dict(case)
    if c["op"] == "clip":
        sizes = [c["big_n"]] * c["big"] + [c["small_n"]] * c["small"]
        width = {"bf16": [2], "f32": [4], "mixed": [2, 4]}[c["act"]]
        # read once, written once
        return {"bytes": sum(2 * n * width[i % len(width)] for i, n in enumerate(sizes)), "flops": 3 * sum(sizes)}
    es = 2 if c["act"] == "bf16" else 4
    B, H, T = c["B"], c["H"], c["T"]
    if c["op"].startswith("conv"):
        d, W = c["d"], c["W"]
        n, par, hist = B * H * T * d, 4 * H * d * (W + bool(c["bias"])), B * H * (W - 1) * d * es
        if c["op"] == "conv_train":
            # x and dy in, y and dx out; the parameters in and their gradients out
            return {"bytes": 4 * n * es + 2 * par + (2 * hist if c["state"] else 0), "flops": n * (8 * W + 12)}
        return {"bytes": 2 * n * es + par + hist * (2 if c["state"] or c["op"] == "conv_step" else 1), "flops": n * (2 * W + 4)}
    G, P, N = c["G"], c["P"], c["N"]
    tok, qk, gate, S = B * H * T * P * es, 2 * B * G * T * N * es, 4 * B * H * T, 4 * B * H * P * N
    first = S if c["state"] or c["op"] == "scan_step" else 0
    # a state of P x N takes one multiply-add a token to update and one to read
    if c["op"] == "scan_train":
        # v, dy, q, k and dt in, and y and all their gradients out; the gradients take the state's and its
        # adjoint's updates and three products with them more
        return {"bytes": 4 * tok + 2 * qk + 2 * gate + S + 2 * first, "flops": 12 * B * H * T * P * N}
    return {"bytes": 2 * tok + qk + gate + S + first, "flops": 4 * B * H * T * P * N}
