"""Cases that measure the sequence-model operators: linear attention with a
decay for each head, the gated norm around a block, and the orthogonalised
update of a weight gradient.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes the inputs of one on the GPU from a seed, ``run()`` makes
one pass, ``work()`` says what a pass cannot do without and ``exact()`` gives
the operator's definition in 64 bits. With ``own`` false a pass is the
operator's plain form in elementary torch operations in 32 bits; with ``own``
true it is the call a user makes of this package.

The block the cases come from: a 1x1 convolution makes queries, keys, values
and gates; linear attention with a decay for each head mixes the tokens; a
gated norm scales what each head gives; a second 1x1 convolution leads back and
the norm after it, its residual scale and the next block's norm join the
residual stream. The weight gradients of the convolutions, and of this
repository's own grouped layers, are orthogonalised before they are applied.
"""
import math

import torch

own = False

CHUNK = 128  # tokens of a chunk in the plain form of the linear attention
NS = (3.4445, -4.7750, 2.0315)  # the quintic of the Newton-Schulz iteration
STEPS = 5
EPS_NORM = 1e-6
EPS_ORTHO = 1e-7
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def _attn(name, do, type_, batch, length, heads, kv_heads, dk, dv, lens="", state=False):
    return {"name": name, "op": "attn", "do": do, "type": type_, "batch": batch, "length": length, "heads": heads,
            "kv_heads": kv_heads, "dk": dk, "dv": dv, "lens": lens, "state": state}


def _step(name, type_, batch, slots, heads, kv_heads, dk, dv):
    return {"name": name, "op": "step", "type": type_, "batch": batch, "slots": slots, "heads": heads, "kv_heads": kv_heads,
            "dk": dk, "dv": dv}


def _norm(name, do, type_, batch, length, dim, gate, act, residual, scale):
    return {"name": name, "op": "norm", "do": do, "type": type_, "batch": batch, "length": length, "dim": dim, "gate": gate,
            "act": act, "residual": residual, "scale": scale}


def _ortho(name, type_, filters, inputs, kernel, groups):
    return {"name": name, "op": "ortho", "type": type_, "filters": filters, "inputs": inputs, "kernel": kernel, "groups": groups}


def listed():
    return [
        # one token of one sequence: the latency of a single decoding step
        _step("step_one", "bf16", 1, 1, 16, 16, 128, 128),
        # a full decoding batch, keys and values shared by four heads, sequences anywhere in the pool of states
        _step("step_batch", "bf16", 256, 320, 16, 4, 128, 128),
        # prompts of different lengths packed into one call, one of them empty, one a single token, each going on from a state
        _attn("prefill_packed", "forward", "bf16", 12, 0, 16, 4, 128, 128, lens="1,1500,17,0,700,64,2000,333,129,1024,65,2360", state=True),
        # the largest: one long prompt
        _attn("prefill_long", "forward", "bf16", 1, 32768, 16, 16, 128, 128),
        # 32 bits throughout, head sizes that fill no tile, a length that ends inside one
        _attn("prefill_fp32_odd", "forward", "fp32", 2, 1111, 6, 3, 72, 96, state=True),
        # a training step's forward and backward with shared keys and values
        _attn("train", "train", "bf16", 4, 4096, 16, 4, 128, 128),
        # the norms around a block for a few decoded tokens: latency
        _norm("norm_few_rows", "forward", "bf16", 8, 1, 4096, "full", "silu", True, True),
        # the same over a prompt
        _norm("norm_prompt", "forward", "bf16", 4, 4096, 4096, "full", "silu", True, True),
        # training in 32 bits on an odd width, one gate a sequence
        _norm("norm_train_odd", "train", "fp32", 6, 683, 1001, "sequence", "sigmoid", True, True),
        # training the gated norm of each head's output: many short rows, no residual
        _norm("norm_train_heads", "train", "bf16", 4, 65536, 128, "full", "silu", False, False),
        # the weight gradient of the fully-connected layer (4096 filters over 256x6x6)
        _ortho("ortho_fc", "fp32", 4096, 256, 6, 1),
        # the weight gradient of the two-group 5x5 layer (256 filters of 48x5x5)
        _ortho("ortho_groups", "fp32", 256, 48, 5, 2),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "step", "norm", "norm", "ortho"))
    type_ = rng.choice(("bf16", "bf16", "fp32"))
    if op in ("attn", "step"):
        kv = rng.choice((1, 2, 3, 4, 8))
        heads = kv * rng.choice((1, 2, 4))
        dk, dv = rng.choice((rng.randint(16, 128), 64, 128)), rng.choice((rng.randint(16, 128), 64, 128))
    if op == "step":
        batch = _log(rng, 1, 256)
        c = _step("", type_, batch, batch + rng.randint(0, 32), heads, kv, dk, dv)
    elif op == "attn":
        do = rng.choice(("forward", "train"))
        most = (32768 * 16 if do == "forward" else 4096 * 64) // heads
        if rng.random() < 0.5:
            count = _log(rng, 1, 16)
            lens = [_log(rng, 1, 2500) if rng.random() > 0.08 else 0 for _ in range(count - 1)] + [_log(rng, 1, 2500)]
            while sum(lens) > most:
                lens = [(n + 1) // 2 for n in lens]
            c = _attn("", do, type_, count, 0, heads, kv, dk, dv, lens=",".join(map(str, lens)), state=rng.random() < 0.5)
        else:
            batch = _log(rng, 1, 8)
            c = _attn("", do, type_, batch, _log(rng, 1, most // batch), heads, kv, dk, dv, state=rng.random() < 0.5)
    elif op == "norm":
        do = rng.choice(("forward", "train"))
        dim = _log(rng, 32, 8192)
        if rng.random() < 0.5:
            dim = max(32, dim // 64 * 64)
        batch = _log(rng, 1, 16)
        length = _log(rng, 1, max(1, (1 << 25) // (dim * batch)))
        c = _norm("", do, type_, batch, length, dim, rng.choice(("none", "full", "sequence")),
                  rng.choice(("none", "sigmoid", "silu")), rng.random() < 0.7, rng.random() < 0.5)
    else:
        kernel = rng.choice((1, 1, 3, 5))
        groups = rng.choice((1, 1, 2, 8, 32))
        most = max(16, 4096 // (kernel * groups))
        c = _ortho("", type_, groups * _log(rng, 4, max(16, 4096 // groups)), _log(rng, 4, most), kernel, groups)
    del c["name"]
    return c


def _lens(case):
    return [int(n) for n in case["lens"].split(",")] if case["lens"] else [case["length"]] * case["batch"]


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    type_ = TYPES[case["type"]]

    def normal(*shape, std=1.0, dtype=type_):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(*shape, dtype=torch.float32):
        return torch.rand(shape, generator=gen, device="cuda").to(dtype)

    s = {"case": case}
    if case["op"] in ("attn", "step"):
        h, hk, dk, dv = case["heads"], case["kv_heads"], case["dk"], case["dv"]
        # half-lives from about two tokens to about a thousand, spread over the heads
        u = (torch.arange(h, device="cuda") + uniform(h)) / h
        s["log_decay"] = -0.35 * torch.exp(-6.0 * u)
        s["scale"] = dk ** -0.5
    if case["op"] == "step":
        b, slots = case["batch"], case["slots"]
        # the three are slices of one projection, as a user's program has them
        qkv = normal(b, h * dk + hk * (dk + dv))
        s["q"] = qkv[:, :h * dk].view(b, h, dk)
        s["k"] = qkv[:, h * dk:(h + hk) * dk].view(b, hk, dk)
        s["v"] = qkv[:, (h + hk) * dk:].view(b, hk, dv)
        s["state"] = normal(slots, h, dk, dv, dtype=torch.float32)
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:b].to(torch.int32)
    elif case["op"] == "attn":
        lens = _lens(case)
        lead = (sum(lens),) if case["lens"] else (case["batch"], case["length"])
        qkv = normal(*lead, h * dk + hk * (dk + dv))
        s["q"] = qkv[..., :h * dk].unflatten(-1, (h, dk))
        s["k"] = qkv[..., h * dk:(h + hk) * dk].unflatten(-1, (hk, dk))
        s["v"] = qkv[..., (h + hk) * dk:].unflatten(-1, (hk, dv))
        s["cu"] = None
        if case["lens"]:
            s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
        s["longest"] = max(lens)
        s["state"] = normal(len(lens), h, dk, dv, dtype=torch.float32) if case["state"] else None
        if case["do"] == "train":
            s["do"] = normal(*lead, h, dv)
            s["dstate"] = normal(len(lens), h, dk, dv, std=0.3, dtype=torch.float32) if case["state"] else None
    elif case["op"] == "norm":
        b, t, d = case["batch"], case["length"], case["dim"]
        s["x"] = normal(b, t, d, std=2.0) if case["residual"] else None
        s["b"] = normal(b, t, d, std=0.7)
        s["gate"] = normal(b, t, d) if case["gate"] == "full" else normal(b, 1, d) if case["gate"] == "sequence" else None
        s["w_post"] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(type_)
        s["scale"] = (0.1 + 0.05 * normal(d, dtype=torch.float32)).to(type_) if case["scale"] else None
        s["w_pre"] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(type_) if case["residual"] else None
        if case["do"] == "train":
            s["dy"] = normal(b, t, d)
            s["dh"] = normal(b, t, d) if case["residual"] else None
    else:
        k, c, r = case["filters"], case["inputs"], case["kernel"]
        n = c * r * r
        # a gradient: a few strong directions and noise of the same energy
        u, v = normal(k, 16, dtype=torch.float32), normal(16, n, std=0.25, dtype=torch.float32)
        s["u"] = ((u @ v + normal(k, n, dtype=torch.float32)) * 1e-3).to(type_).view(k, c, r, r)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import grouped_convolution_amd as G
        if op == "step":
            o = G.gconv_linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"], slots=s["slots"])
            return {"o": o, "state": s["state"]}
        if op == "attn":
            kw = dict(scale=s["scale"], cu_seqlens=s["cu"], initial_state=s["state"])
            o, final = G.gconv_linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], **kw)
            out = {"o": o, "final": final}
            if case["do"] == "train":
                dq, dk, dv, ds = G.gconv_linattn_bwd(s["do"], s["q"], s["k"], s["v"], s["log_decay"], d_final_state=s["dstate"], **kw)
                out.update(dq=dq, dk=dk, dv=dv)
                if ds is not None:
                    out["dstate"] = ds
            return out
        if op == "norm":
            kw = dict(gate=s["gate"], act=case["act"], w_post=s["w_post"], scale=s["scale"], w_pre=s["w_pre"], eps=EPS_NORM)
            y, h = G.gconv_normgate_fwd(s["x"], s["b"], **kw)
            out = {"y": y, "h": h}
            if case["do"] == "train":
                names = ("dx", "db", "dgate", "dw_post", "dscale", "dw_pre")
                out.update(zip(names, G.gconv_normgate_bwd(s["dy"], s["dh"], s["x"], s["b"], **kw)))
            return {k: v for k, v in out.items() if v is not None}
        return G.gconv_orthogonalize(s["u"], groups=case["groups"], steps=STEPS, eps=EPS_ORTHO)
    if op == "step":
        return _plain_step(s)
    if op == "attn":
        return _plain_attn(s)
    if op == "norm":
        return _plain_norm(s)
    return _plain_ortho(s)


def _plain_step(s):
    rep = s["q"].shape[1] // s["k"].shape[1]
    q, k, v = s["q"].float(), s["k"].float().repeat_interleave(rep, 1), s["v"].float().repeat_interleave(rep, 1)
    new = s["state"][s["slots"]] * torch.exp(s["log_decay"])[:, None, None] + k[..., None] * v[..., None, :]
    s["state"][s["slots"]] = new
    o = (q[..., None, :] @ new)[..., 0, :] * s["scale"]
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _plain_linattn(q, k, v, g, scale, state, before, lens):
    """Linear attention of [N, T, H, D] whose sequences end at T (T a multiple of CHUNK; k is 0 before them);
    before [N, T]: tokens of the sequence up to and with each. Returns o and the final state."""
    n, t, h, dk = q.shape
    rep = h // k.shape[2]
    k, v = k.repeat_interleave(rep, 2), v.repeat_interleave(rep, 2)
    c = t // CHUNK
    qc, kc, vc = (x.unflatten(1, (c, CHUNK)).permute(0, 3, 1, 2, 4) for x in (q * scale, k, v))  # [N, H, c, CHUNK, D]
    i = torch.arange(CHUNK, device=q.device, dtype=torch.float32)
    j = torch.arange(c, device=q.device, dtype=torch.float32)
    g = g[:, None, None]
    near = i[:, None] - i
    far = j[:, None] - j - 1
    within = torch.where(near >= 0, torch.exp(g * near.clamp(min=0)), 0.0)[:, None]
    across = torch.where(far >= 0, torch.exp(g * CHUNK * far.clamp(min=0)), 0.0)
    o = (qc @ kc.mT * within) @ vc
    left = (kc * torch.exp(g * (CHUNK - 1 - i)[:, None])[:, None]).mT @ vc  # what each chunk leaves behind
    flat = left.flatten(3)
    o = o + (qc * torch.exp(g * (i + 1)[:, None])[:, None]) @ (across @ flat).unflatten(3, left.shape[3:])
    final = (torch.exp(g[:, 0] * CHUNK * (c - 1 - j))[:, None] @ flat).unflatten(3, left.shape[3:])[:, :, 0]
    o = o.permute(0, 2, 3, 1, 4).flatten(1, 2)
    if state is not None:
        g = g[:, 0, 0]
        decayed = q * scale * torch.exp(before.clamp(min=0)[..., None] * g)[..., None]
        o = o + (decayed.transpose(1, 2) @ state).transpose(1, 2)
        final = final + state * torch.exp(lens[:, None] * g)[..., None, None]
    return o, final


def _plain_attn(s):
    case, cu = s["case"], s["cu"]
    train = case["do"] == "train"
    leaves = [s[n].float() for n in ("q", "k", "v")] + ([s["state"]] if s["state"] is not None else [])
    if train:
        leaves = [x.detach().requires_grad_() for x in leaves]
    q, k, v = leaves[:3]
    state = leaves[3] if len(leaves) > 3 else None
    t = -(-max(s["longest"], 1) // CHUNK) * CHUNK
    col = torch.arange(t, device=q.device)
    with torch.set_grad_enabled(train):
        if cu is not None:
            # every sequence moved to the end of a row of its own
            lens = (cu[1:] - cu[:-1]).long()
            at = cu[1:, None] - t + col
            valid = at >= cu[:-1, None]
            at = torch.where(valid, at, 0).clamp(max=q.shape[0] - 1)
            q, k, v = (torch.where(valid[..., None, None], x[at], 0.0) for x in (q, k, v))
        else:
            lens = torch.full((q.shape[0],), q.shape[1], device=q.device)
            q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, t - x.shape[1], 0)) for x in (q, k, v))
        before = (col + 1 - t + lens[:, None]).float()
        o, final = _plain_linattn(q, k, v, s["log_decay"], s["scale"], state, before, lens.float())
        if cu is not None:
            token = torch.arange(leaves[0].shape[0], device=q.device)
            seq = torch.searchsorted(cu, token.to(cu.dtype), right=True) - 1
            o = o[seq, t + token - cu[1:][seq]]
        else:
            o = o[:, t - leaves[0].shape[1]:]
    out = {"o": o.detach().to(s["q"].dtype), "final": final.detach()}
    if train:
        grads = [s["do"].float()] + ([s["dstate"]] if state is not None else [])
        got = torch.autograd.grad([o, final][:len(grads)], leaves, grads)
        out.update(zip(("dq", "dk", "dv"), (x.to(s["q"].dtype) for x in got)))
        if state is not None:
            out["dstate"] = got[3]
    return out


def _act(x, act):
    return x if act == "none" else torch.sigmoid(x) if act == "sigmoid" else x * torch.sigmoid(x)


def _plain_norm(s):
    case = s["case"]
    train = case["do"] == "train"
    names = [n for n in ("x", "b", "gate", "w_post", "scale", "w_pre") if s[n] is not None]
    leaf = {n: s[n].float().detach().requires_grad_(train) for n in names}
    with torch.set_grad_enabled(train):
        b = leaf["b"]
        y = b * torch.rsqrt(b.square().mean(-1, keepdim=True) + EPS_NORM) * leaf["w_post"]
        if "gate" in leaf:
            y = y * _act(leaf["gate"], case["act"])
        if "scale" in leaf:
            y = y * leaf["scale"]
        if "x" in leaf:
            y = y + leaf["x"]
        outs = [y]
        if "w_pre" in leaf:
            outs.append(y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS_NORM) * leaf["w_pre"])
    out = dict(zip(("y", "h"), (v.detach().to(s["b"].dtype) for v in outs)))
    if train:
        grads = torch.autograd.grad(outs, list(leaf.values()), [s["dy"].float(), s["dh"].float()] if len(outs) > 1 else [s["dy"].float()])
        out.update(("d" + n, v.to(s[n].dtype)) for n, v in zip(names, grads))
    return out


def _plain_ortho(s):
    u = s["u"]
    x = u.float().reshape(s["case"]["groups"], -1, u[0].numel())
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.mT
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS_ORTHO)
    for _ in range(STEPS):
        a = x @ x.mT
        x = NS[0] * x + (NS[1] * a + NS[2] * (a @ a)) @ x
    return (x.mT if tall else x).reshape(u.shape).to(torch.bfloat16)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 4 if case["type"] == "fp32" else 2
    if case["op"] in ("attn", "step"):
        h, hk, dk, dv = case["heads"], case["kv_heads"], case["dk"], case["dv"]
    if case["op"] == "step":
        b = case["batch"]
        return {"bytes": b * (size * (h * (dk + dv) + hk * (dk + dv)) + 8 * h * dk * dv), "flops": 5.0 * b * h * dk * dv}
    if case["op"] == "attn":
        lens = _lens(case)
        total, states = sum(lens), len(lens) * h * dk * dv * 4
        token = size * (h * (dk + dv) + hk * (dk + dv))
        # q, k, v read and o written, the final states written; training also reads do and writes dq, dk and dv
        moved = total * token + states * (2 if case["state"] else 1)
        # the recurrence: one update of the state and one product with it for each token and head
        flops = 4.0 * total * h * dk * dv
        if case["do"] == "train":
            moved += total * (token + size * h * dv) + (2 * states if case["state"] else 0)
            flops += 10.0 * total * h * dk * dv
        return {"bytes": moved, "flops": flops}
    if case["op"] == "norm":
        rows, d = case["batch"] * case["length"], case["dim"]
        gate = {"none": 0, "full": rows, "sequence": case["batch"]}[case["gate"]]
        wide = (3 if case["residual"] else 1) * rows + rows + gate  # x, h and y or y alone; b; the gate
        if case["do"] == "train":
            wide += (3 if case["residual"] else 1) * rows + rows + gate  # dy, dh, dx or dy alone; db; dgate
        return {"bytes": size * d * wide, "flops": (12.0 if case["do"] == "forward" else 45.0) * rows * d}
    m, n = case["filters"] // case["groups"], case["inputs"] * case["kernel"] ** 2
    total = case["groups"] * m * n
    m, n = min(m, n), max(m, n)
    # each step: a Gram matrix and its square, of which half is enough, and a product with the iterate
    return {"bytes": total * (size + 2), "flops": STEPS * case["groups"] * (1.0 * m * m * n + 1.0 * m * m * m + 2.0 * m * m * n)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "step":
            return _exact_step(s)
        if case["op"] == "attn":
            return _exact_attn(s)
        if case["op"] == "norm":
            return _exact_norm(s)
        return _exact_ortho(s)


def _exact_step(s):
    state = s["state"].double()
    h, hk = s["q"].shape[1], s["k"].shape[1]
    head = torch.arange(h, device="cuda") // (h // hk)
    o = torch.empty(s["q"].shape[0], h, s["v"].shape[2], dtype=torch.float64, device="cuda")
    keep = s["log_decay"].double().exp()
    for i, slot in enumerate(s["slots"].tolist()):
        new = keep.view(-1, 1, 1) * state[slot] + torch.einsum("hd,he->hde", s["k"][i].double()[head], s["v"][i].double()[head])
        o[i] = torch.einsum("hd,hde->he", s["q"][i].double(), new) * s["scale"]
        state[slot] = new
    return {"o": o, "state": state}


def _exact_attn(s):
    """The sum over all earlier tokens, a block of rows at a time, one sequence and one head after another."""
    case = s["case"]
    h, hk, dk, dv = case["heads"], case["kv_heads"], case["dk"], case["dv"]
    train, lens = case["do"] == "train", _lens(case)
    f64 = dict(dtype=torch.float64, device="cuda")
    q, k, v = (s[n].reshape(-1, *s[n].shape[-2:]).double() for n in ("q", "k", "v"))
    out = {"o": torch.zeros(q.shape[0], h, dv, **f64), "final": torch.zeros(len(lens), h, dk, dv, **f64)}
    if train:
        do = s["do"].reshape(-1, h, dv).double()
        out.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
        if s["state"] is not None:
            out["dstate"] = torch.zeros(len(lens), h, dk, dv, **f64)
    first = 0
    for n, size in enumerate(lens):
        rows = slice(first, first + size)
        first += size
        place = torch.arange(size, **f64)
        for head in range(h):
            g, kh = s["log_decay"][head].double(), head // (h // hk)
            qs, ks, vs = q[rows, head] * s["scale"], k[rows, kh], v[rows, kh]
            s0 = s["state"][n, head].double() if s["state"] is not None else torch.zeros(dk, dv, **f64)
            ds = s["dstate"][n, head].double() if train and s["state"] is not None else torch.zeros(dk, dv, **f64)
            decay = torch.exp(g * (place + 1))[:, None]    # of the state before the sequence, at each token
            rest = torch.exp(g * (size - 1 - place))[:, None]  # of each token, at the sequence's end
            end = torch.exp(g * size)
            out["final"][n, head] = (ks * rest).T.contiguous() @ vs + end * s0
            step = max(1, min(size, (1 << 26) // max(size, 1)))
            for a in range(0, size, step):
                b = min(size, a + step)
                w = torch.exp(g * (place[a:b, None] - place[None, :b]).clamp(min=0)).tril(a)
                p = qs[a:b] @ ks[:b].T.contiguous() * w
                out["o"][rows, head][a:b] = p @ vs[:b] + decay[a:b] * (qs[a:b] @ s0)
                if train:
                    d = do[rows, head][a:b]
                    dp = d @ vs[:b].T.contiguous() * w
                    out["dq"][rows, head][a:b] = s["scale"] * (dp @ ks[:b] + decay[a:b] * (d @ s0.T.contiguous()))
                    out["dk"][rows, kh][:b] += dp.T.contiguous() @ qs[a:b]
                    out["dv"][rows, kh][:b] += p.T.contiguous() @ d
            if train:
                out["dk"][rows, kh] += rest * (vs @ ds.T.contiguous())
                out["dv"][rows, kh] += rest * (ks @ ds)
                if s["state"] is not None:
                    out["dstate"][n, head] = end * ds + (qs * decay).T.contiguous() @ do[rows, head]
    for name in ("o", "dq", "dk", "dv"):
        if name in out:
            out[name] = out[name].reshape(s["q" if name in ("o", "dq") else name[1]].shape[:-1] + (out[name].shape[-1],))
    return out


def _exact_norm(s):
    case = s["case"]
    d = case["dim"]
    flat = lambda n: s[n].expand_as(s["b"]).reshape(-1, d).double() if s[n] is not None else None  # noqa: E731
    one = torch.ones(d, dtype=torch.float64, device="cuda")
    vec = lambda n: s[n].double() if s[n] is not None else one  # noqa: E731
    x, b, z = flat("x"), flat("b"), flat("gate")
    rb = (torch.linalg.vector_norm(b, dim=1, keepdim=True) ** 2 / d + EPS_NORM) ** -0.5
    sig = 1 / (1 + torch.exp(-z)) if z is not None else None
    if z is None:
        a, da = torch.ones_like(b), None
    elif case["act"] == "none":
        a, da = z, torch.ones_like(z)
    elif case["act"] == "sigmoid":
        a, da = sig, sig * (1 - sig)
    else:
        a, da = z * sig, sig + z * sig * (1 - sig)
    bn = b * rb
    n = bn * vec("w_post")
    y = vec("scale") * a * n + (x if x is not None else 0)
    shape = s["b"].shape
    out = {"y": y.view(shape)}
    if s["w_pre"] is not None:
        ry = (torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / d + EPS_NORM) ** -0.5
        yn = y * ry
        out["h"] = (yn * s["w_pre"].double()).view(shape)
    if case["do"] != "train":
        return out
    dy = s["dy"].reshape(-1, d).double()
    if s["w_pre"] is not None:
        dh = s["dh"].reshape(-1, d).double()
        e = dh * s["w_pre"].double()
        dy = dy + ry * (e - yn * (e * yn).mean(1, keepdim=True))
    if x is not None:
        out["dx"] = dy.view(shape)
    du = dy * vec("scale")
    e = du * a * vec("w_post")
    out["db"] = (rb * (e - bn * (e * bn).mean(1, keepdim=True))).view(shape)
    if z is not None:
        dz = du * n * da
        out["dgate"] = (dz if case["gate"] == "full" else dz.view(case["batch"], -1, d).sum(1)).view(s["gate"].shape)
    out["dw_post"] = (du * a * bn).sum(0)
    if s["scale"] is not None:
        out["dscale"] = (dy * a * n).sum(0)
    if s["w_pre"] is not None:
        out["dw_pre"] = (dh * yn).sum(0)
    return out


def _exact_ortho(s):
    u = s["u"]
    out = []
    for m in u.double().reshape(u.shape[0], -1).chunk(s["case"]["groups"]):
        wide = m.shape[0] <= m.shape[1]
        m = m if wide else m.T.contiguous()
        m = m / (torch.linalg.vector_norm(m) + EPS_ORTHO)
        for _ in range(STEPS):
            gram = m @ m.T.contiguous()
            m = NS[0] * m + NS[1] * (gram @ m) + NS[2] * (gram @ (gram @ m))
        out.append(m if wide else m.T)
    return torch.cat(out).reshape(u.shape)
