"""Cases that measure the operators of a token model: the short causal
convolution and the selective state space scan that mix the tokens in a block,
and the two ends at which a model meets its tokens, the embedding and the
softmax cross entropy against the vocabulary.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes the inputs of one on the GPU from a seed, ``run()`` makes
one pass, ``work()`` says what a pass cannot do without and ``exact()`` gives
the operator's definition in 64 bits. With ``own`` false a pass is the
operator's plain form in elementary torch operations in 32 bits; with ``own``
true it is the call a user makes of this package.

The block the cases come from: tokens are embedded; a 1x1 convolution makes a
block's inputs, a short causal convolution joins each channel's last tokens, a
scan whose decay depends on the token mixes them over any distance, a gate and
a second 1x1 convolution lead back; at the end the loss of the next token is
taken against the whole vocabulary.
"""
import math

import torch

own = False

CHUNK = 64  # tokens of a chunk in the plain form of the scan
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
INDEX = {"i32": torch.int32, "i64": torch.int64}
IGNORED = -100  # a target that does not count


# ---------------------------------------------------------------- the cases

def _conv(name, do, type_, batch, length, dim, taps, act, bias, lens="", state=False):
    return {"name": name, "op": "conv", "do": do, "type": type_, "batch": batch, "length": length, "dim": dim, "taps": taps,
            "act": act, "bias": bias, "lens": lens, "state": state}


def _scan(name, do, type_, batch, length, dim, states, groups, gate, lens="", state=False):
    return {"name": name, "op": "scan", "do": do, "type": type_, "batch": batch, "length": length, "dim": dim, "states": states,
            "groups": groups, "gate": gate, "lens": lens, "state": state}


def _embed(name, do, type_, index, tokens, rows, dim, padded):
    return {"name": name, "op": "embed", "do": do, "type": type_, "index": index, "tokens": tokens, "rows": rows, "dim": dim,
            "padded": padded}


def _xent(name, do, type_, index, tokens, vocab, dim, ignored, lse):
    return {"name": name, "op": "xent", "do": do, "type": type_, "index": index, "tokens": tokens, "vocab": vocab, "dim": dim,
            "ignored": ignored, "lse": lse}


def listed():
    return [
        # a decoding batch takes in one token each: latency
        _conv("conv_step", "step", "bf16", 64, 80, 4096, 4, "silu", True),
        # prompts of different lengths in one call, in 32 bits, on a width that fills no piece, each going on from a state
        _conv("conv_packed_fp32", "forward", "fp32", 9, 0, 1001, 3, "silu", True, lens="700,1,0,2,1500,333,17,2000,64", state=True),
        # a training step's convolution
        _conv("conv_train", "train", "bf16", 4, 4096, 4096, 4, "silu", True),
        # a full decoding batch, sequences anywhere in the pool of states
        _scan("scan_step", "step", "bf16", 256, 320, 4096, 16, 1, True),
        # prompts of different lengths packed into one call, one of them empty, one a single token, each going on from a state
        _scan("scan_packed", "forward", "bf16", 10, 0, 4096, 16, 1, True, lens="1,1500,17,0,700,64,2000,333,129,1024", state=True),
        # one long prompt
        _scan("scan_long", "forward", "bf16", 1, 32768, 2048, 16, 1, True),
        # a training step's forward and backward
        _scan("scan_train", "train", "bf16", 4, 2048, 4096, 16, 1, True),
        # 32 bits throughout, widths and lengths that fill no tile, two groups of inputs and outputs
        _scan("scan_train_fp32_odd", "train", "fp32", 3, 613, 300, 10, 2, False, state=True),
        # the embedding of a few decoded tokens: latency
        _embed("embed_few", "forward", "fp32", "i32", 8, 32000, 4096, False),
        # a training step's embedding and its gradient, some frequent tokens and many that do not occur
        _embed("embed_train", "train", "bf16", "i64", 16384, 50001, 2048, True),
        # the largest: the loss of a training step and its gradients
        _xent("xent_train", "train", "bf16", "i64", 8192, 65536, 2048, 0.05, False),
        # the same in 32 bits, with sizes that fill no tile and a term on the normaliser
        _xent("xent_train_fp32_odd", "train", "fp32", "i32", 501, 10007, 1000, 0.2, True),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _packed(rng, longest, most):
    count = _log(rng, 1, 16)
    lens = [_log(rng, 1, longest) if rng.random() > 0.08 else 0 for _ in range(count - 1)] + [_log(rng, 1, longest)]
    while sum(lens) > most or count * max(lens) > 2 * most:
        lens = [(n + 1) // 2 for n in lens]
    return count, ",".join(map(str, lens))


def draw(rng):
    op = rng.choice(("conv", "scan", "scan", "embed", "xent"))
    type_ = rng.choice(("bf16", "bf16", "fp32"))
    index = rng.choice(("i32", "i64"))
    if op == "conv":
        do = rng.choice(("step", "forward", "train", "train"))
        dim = _log(rng, 16, 8192)
        dim = max(16, dim // 64 * 64) if rng.random() < 0.6 else dim
        most = (1 << 26) // dim
        kw = dict(type_=type_, dim=dim, taps=rng.choice((2, 3, 4, 4, rng.randint(1, 8))), act=rng.choice(("none", "silu", "silu")),
                  bias=rng.random() < 0.7)
        if do == "step":
            batch = _log(rng, 1, 512)
            c = _conv("", do, batch=batch, length=batch + rng.randint(0, 64), **kw)
        elif rng.random() < 0.5:
            count, lens = _packed(rng, 2500, min(most, 16384))
            c = _conv("", do, batch=count, length=0, lens=lens, state=rng.random() < 0.5, **kw)
        else:
            batch = _log(rng, 1, 8)
            c = _conv("", do, batch=batch, length=_log(rng, 1, min(16384, most // batch)), state=rng.random() < 0.5, **kw)
    elif op == "scan":
        do = rng.choice(("step", "forward", "train", "train"))
        states = rng.choice((16, 16, 16, 8, 32, 64, rng.randint(1, 64)))
        groups = rng.choice((1, 1, 2, 4))
        dim = _log(rng, 32, 4096)
        dim = max(64, dim // 64 * 64) if rng.random() < 0.6 else max(4, dim // groups) * groups
        most = (1 << 30 if do == "forward" else 1 << 29) // (dim * states)
        kw = dict(type_=type_, dim=dim, states=states, groups=groups, gate=rng.random() < 0.7)
        if do == "step":
            batch = _log(rng, 1, 256)
            c = _scan("", do, batch=batch, length=batch + rng.randint(0, 64), **kw)
        elif rng.random() < 0.5:
            count, lens = _packed(rng, 2500, min(most, 8192))
            c = _scan("", do, batch=count, length=0, lens=lens, state=rng.random() < 0.5, **kw)
        else:
            batch = _log(rng, 1, 8)
            c = _scan("", do, batch=batch, length=_log(rng, 1, min(32768 if do == "forward" else 8192, most) // batch),
                      state=rng.random() < 0.5, **kw)
    elif op == "embed":
        dim = _log(rng, 16, 8192)
        dim = max(16, dim // 64 * 64) if rng.random() < 0.7 else dim
        rows = _log(rng, 100, min(150000, (1 << 29) // dim))
        c = _embed("", rng.choice(("forward", "train", "train")), type_, index, _log(rng, 1, min(65536, (1 << 27) // dim)), rows, dim,
                   rng.random() < 0.5)
    else:
        do = rng.choice(("forward", "train", "train"))
        dim = _log(rng, 32, 4096)
        dim = max(64, dim // 64 * 64) if rng.random() < 0.7 else dim
        vocab = _log(rng, 50, min(150000, (1 << 28) // dim))
        most = (1 << (40 if type_ == "bf16" else 37)) // (dim * vocab)
        c = _xent("", do, type_, index, _log(rng, 1, max(1, min(8192, most, (1 << 29) // vocab))), vocab, dim, rng.choice((0.0, 0.1, 0.5)),
                  do == "train" and rng.random() < 0.3)
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

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    def words(count, most, dtype):
        # token numbers as in a text: the r-th most frequent one about 1/r as often as the first
        rank = torch.exp(uniform(count) * math.log(most)).long().clamp(1, most) - 1
        return torch.randperm(most, generator=gen, device="cuda")[rank].to(dtype)

    s = {"case": case}
    step, train = case["do"] == "step", case["do"] == "train"
    if case["op"] in ("conv", "scan"):
        d = case["dim"]
        lens = [] if step else _lens(case)
        lead = (case["batch"],) if step else (sum(lens),) if case["lens"] else (case["batch"], case["length"])
        s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if case["lens"] else None
        s["longest"] = max(lens, default=1)
        s["slots"] = None
        if step:
            s["slots"] = torch.randperm(case["length"], generator=gen, device="cuda")[:case["batch"]].to(torch.int32)
        pool = case["length"] if step else len(lens)
    if case["op"] == "conv":
        k = case["taps"]
        # the convolution's inputs are the first half of what a projection gives, the gates the second
        s["x"] = normal(*lead, 2 * d)[..., :d]
        s["w"] = normal(d, k, std=k ** -0.5)
        s["bias"] = normal(d, std=0.2) if case["bias"] else None
        s["state"] = normal(pool, k - 1, d) if step or case["state"] else None
        if train:
            s["dy"] = normal(*lead, d)
            s["dstate"] = normal(pool, k - 1, d, std=0.3) if case["state"] else None
    elif case["op"] == "scan":
        n, g = case["states"], case["groups"]
        s["u"] = torch.nn.functional.silu(normal(*lead, d).float()).to(type_)
        # steps from about 0.001 to 0.1, spread over the channels and moved by the tokens
        first = torch.exp(uniform(d, lo=math.log(0.001), hi=math.log(0.1)))
        s["dt_bias"] = torch.log(torch.expm1(first))
        s["dt"] = normal(*lead, d, std=0.7)
        # the two are slices of one projection, as a user's program has them
        bc = normal(*lead, 8 + 2 * g * n)
        s["b"] = bc[..., 8:8 + g * n].unflatten(-1, (g, n))
        s["c"] = bc[..., 8 + g * n:].unflatten(-1, (g, n))
        s["a"] = -torch.arange(1, n + 1, device="cuda") * torch.exp(0.2 * normal(d, n, dtype=torch.float32))
        s["skip"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        s["gate"] = normal(*lead, 2 * d)[..., d:] if case["gate"] else None
        s["state"] = normal(pool, d, n, std=0.5, dtype=torch.float32) if step or case["state"] else None
        if train:
            s["dy"] = normal(*lead, d)
            s["dstate"] = normal(pool, d, n, std=0.3, dtype=torch.float32) if case["state"] else None
    elif case["op"] == "embed":
        s["ids"] = words(case["tokens"], case["rows"], INDEX[case["index"]])
        if case["padded"]:
            s["ids"][uniform(case["tokens"]) < 0.1] = -1
        s["table"] = normal(case["rows"], case["dim"], std=0.02)
        s["scale"] = case["dim"] ** 0.5
        if train:
            s["dy"] = normal(case["tokens"], case["dim"], std=1e-3)
    else:
        m, v, d = case["tokens"], case["vocab"], case["dim"]
        s["h"] = normal(m, d)
        s["w"] = normal(v, d, std=2 * d ** -0.5)
        s["targets"] = words(m, v, INDEX[case["index"]])
        s["targets"][uniform(m) < case["ignored"]] = IGNORED
        s["scale"] = 0.8
        if train:
            # a mean over the tokens, some of them weighted
            s["dloss"] = uniform(m, lo=0.5, hi=1.5) / m
            s["dlse"] = uniform(m, lo=0.0, hi=1e-2) / m if case["lse"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op, train = case["op"], case["do"] == "train"
    if not own:
        return {"conv": _plain_conv, "scan": _plain_scan, "embed": _plain_embed, "xent": _plain_xent}[op](s)
    import grouped_convolution_amd as G
    if op == "conv":
        if case["do"] == "step":
            y = G.gconv_shortconv_step(s["x"], s["w"], s["state"], s["bias"], act=case["act"], slots=s["slots"])
            return {"y": y, "state": s["state"]}
        kw = dict(act=case["act"], cu_seqlens=s["cu"], initial_state=s["state"])
        y, final = G.gconv_shortconv_fwd(s["x"], s["w"], s["bias"], **kw)
        out = {"y": y, "final": final}
        if train:
            names = ("dx", "dw", "dbias", "dstate")
            out.update(zip(names, G.gconv_shortconv_bwd(s["dy"], s["x"], s["w"], s["bias"], d_final_state=s["dstate"], **kw)))
    elif op == "scan":
        args = [s[n] for n in ("u", "dt", "a", "b", "c")]
        kw = dict(skip=s["skip"], gate=s["gate"], dt_bias=s["dt_bias"], softplus=True)
        if case["do"] == "step":
            y = G.gconv_scan_step(*args, s["state"], slots=s["slots"], **kw)
            return {"y": y, "state": s["state"]}
        kw.update(cu_seqlens=s["cu"], initial_state=s["state"])
        y, final = G.gconv_scan_fwd(*args, **kw)
        out = {"y": y, "final": final}
        if train:
            names = ("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dstate")
            out.update(zip(names, G.gconv_scan_bwd(s["dy"], *args, d_final_state=s["dstate"], **kw)))
    elif op == "embed":
        out = {"y": G.gconv_embed_fwd(s["table"], s["ids"], scale=s["scale"])}
        if train:
            out["dtable"] = G.gconv_embed_bwd(s["dy"], s["ids"], case["rows"], scale=s["scale"])
    else:
        loss, lse = G.gconv_xent_fwd(s["h"], s["w"], s["targets"], scale=s["scale"])
        out = {"loss": loss, "lse": lse}
        if train:
            grads = G.gconv_xent_bwd(s["dloss"], s["h"], s["w"], s["targets"], lse, dlse=s["dlse"], scale=s["scale"])
            out.update(zip(("dh", "dw"), grads))
    return {k: v for k, v in out.items() if v is not None}


def _places(s, count):
    """For each of `count` packed tokens (or those of a batch, one sequence after another): its sequence, its place in that,
    and the sequences' lengths."""
    case = s["case"]
    token = torch.arange(count, device="cuda")
    if s["cu"] is None:
        return token // case["length"], token % case["length"], torch.full((case["batch"],), case["length"], device="cuda")
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, token, right=True) - 1
    return seq, token - cu[seq], cu[1:] - cu[:-1]


def _silu_grad(x):
    sig = torch.sigmoid(x)
    return sig * (1 + x * (1 - sig))


def _plain_conv(s):
    case = s["case"]
    k, d, type_ = case["taps"], case["dim"], s["x"].dtype
    w, silu = s["w"].float(), case["act"] == "silu"
    bias = s["bias"].float() if s["bias"] is not None else 0.0
    if case["do"] == "step":
        slots = s["slots"].long()
        window = torch.cat([s["state"][slots], s["x"][:, None]], 1)
        p = (window.float() * w.T).sum(1) + bias
        s["state"][slots] = window[:, 1:]
        return {"y": (p * torch.sigmoid(p) if silu else p).to(type_), "state": s["state"]}
    x = s["x"].reshape(-1, d).float()
    count = x.shape[0]
    seq, place, lens = _places(s, count)
    state = s["state"].float() if s["state"] is not None else torch.zeros(len(lens), k - 1, d, device="cuda")
    token = torch.arange(count, device="cuda")

    def back(j):  # each token's input j places before it
        if j == 0:
            return x
        near = x[(token - j).clamp(min=0)]
        return torch.where((place >= j)[:, None], near, state[seq, (k - 1 - j + place).clamp(max=k - 2)])

    p = sum(w[:, k - 1 - j] * back(j) for j in range(k)) + bias
    y = p * torch.sigmoid(p) if silu else p
    first = lens.cumsum(0) - lens
    i = torch.arange(k - 1, device="cuda")
    at = lens[:, None] - (k - 1) + i  # the places that a sequence leaves behind
    held = torch.where((at >= 0)[..., None], x[(first[:, None] + at).clamp(0, max(count - 1, 0))],
                       state.gather(1, (at + k - 1).clamp(max=max(k - 2, 0))[..., None].expand(-1, -1, d)))
    out = {"y": y.to(type_).view(s["x"].shape), "final": held.to(type_)}
    if case["do"] == "train":
        dp = s["dy"].reshape(-1, d).float()
        if silu:
            dp = dp * _silu_grad(p)
        size = lens[seq]
        dx = torch.zeros_like(x)
        for j in range(k):
            inside = (place + j < size)[:, None]
            dx += w[:, k - 1 - j] * torch.where(inside, dp[(token + j).clamp(max=count - 1)], 0.0)
        dstate = torch.zeros(len(lens), k - 1, d, device="cuda")
        for i in range(k - 1):
            for j in range(k - 1 - i, k):  # the place of the token that reads it: i - (k - 1) + j
                to = i - (k - 1) + j
                reads = (lens > to)[:, None]
                dstate[:, i] += w[:, k - 1 - j] * torch.where(reads, dp[(first + to).clamp(max=count - 1)], 0.0)
        if s["dstate"] is not None:
            left = s["dstate"].float()
            inside = at >= 0
            dx[(first[:, None] + at)[inside]] += left[inside]
            n = torch.arange(len(lens), device="cuda")[:, None].expand(-1, k - 1)
            dstate[n[~inside], (at + k - 1)[~inside]] += left[~inside]
        out["dx"] = dx.to(type_).view(s["x"].shape)
        out["dw"] = torch.stack([(dp * back(k - 1 - j)).sum(0) for j in range(k)], 1).to(type_)
        if s["bias"] is not None:
            out["dbias"] = dp.sum(0).to(type_)
        if s["state"] is not None:
            out["dstate"] = dstate.to(type_)
    return out


def _recurrence(a, b, start):
    """h_t = a_t h_{t-1} + b_t along axis 1 from h_{-1} = start; a [N, T, ...] and b are overwritten, b becomes h."""
    n, t = a.shape[:2]
    for j0 in range(0, t, CHUNK * (t // CHUNK) or t):
        # the whole chunks side by side, then what is left as one of its own
        size = CHUNK if t - j0 >= CHUNK else t - j0
        count = (t - j0) // size
        ac, bc = (x[:, j0:j0 + count * size].unflatten(1, (count, size)) for x in (a, b))
        for i in range(1, size):
            bc[:, :, i] += ac[:, :, i] * bc[:, :, i - 1]
            ac[:, :, i] *= ac[:, :, i - 1]
        for c in range(count):
            bc[:, c] += ac[:, c] * start[:, None]
            start = bc[:, c, -1]
    return b


def _plain_scan(s):
    case = s["case"]
    d, n, g, type_ = case["dim"], case["states"], case["groups"], s["u"].dtype
    rep = d // g
    dt = s["dt"].float() + s["dt_bias"]
    raw, u, a = dt, s["u"].float(), s["a"]
    dt = torch.nn.functional.softplus(dt, threshold=1e9)
    b, c = s["b"].float(), s["c"].float()
    z = s["gate"].float() if s["gate"] is not None else None
    if case["do"] == "step":
        b, c = b.repeat_interleave(rep, 1), c.repeat_interleave(rep, 1)
        slots = s["slots"].long()
        h = s["state"][slots] * torch.exp(dt[..., None] * a) + (dt * u)[..., None] * b
        s["state"][slots] = h
        y = (h * c).sum(-1) + s["skip"] * u
        return {"y": (y * (z * torch.sigmoid(z)) if z is not None else y).to(type_), "state": s["state"]}
    shape = u.shape
    if s["cu"] is not None:
        # every sequence moved to a row of its own; places past its end take no step
        cu = s["cu"].long()
        lens = cu[1:] - cu[:-1]
        at = cu[:-1, None] + torch.arange(s["longest"], device="cuda")
        valid = at < cu[1:, None]
        at = at.clamp(max=u.shape[0] - 1)

        def rows(x):
            return torch.where(valid.view(valid.shape + (1,) * (x.dim() - 1)), x[at], 0.0)

        def tokens(x):
            return x[valid]
    else:
        rows = tokens = lambda x: x  # noqa: E731
    dt, raw, u, b, c = (rows(x) for x in (dt, raw, u, b, c))
    z = rows(z) if z is not None else None
    wide = lambda x: x.repeat_interleave(rep, 2)  # noqa: E731
    state = s["state"] if s["state"] is not None else torch.zeros(u.shape[0], d, n, device="cuda")
    decay = torch.exp(dt[..., None] * a)
    h = _recurrence(decay.clone(), (dt * u)[..., None] * wide(b), state)
    y = (h * wide(c)).sum(-1) + s["skip"] * u
    final = h[:, -1].clone() if h.shape[1] else state.clone()
    out = {"y": tokens(y * (z * torch.sigmoid(z)) if z is not None else y).to(type_).view(shape), "final": final}
    if case["do"] != "train":
        return out
    dy = rows(s["dy"].float())
    if z is not None:
        out["dgate"] = tokens(dy * y * _silu_grad(z)).to(type_).view(shape)
        dy = dy * (z * torch.sigmoid(z))
    del y
    dc = (dy[..., None] * h).unflatten(2, (g, rep)).sum(3)
    # the adjoint state runs the other way: g_t = c_t dy_t + decay_{t+1} g_{t+1}
    back = torch.ones_like(decay)
    back[:, 1:] = decay[:, 1:].flip(1)
    start = s["dstate"] if s["dstate"] is not None else torch.zeros_like(state)
    adj = _recurrence(back, (dy[..., None] * wide(c)).flip(1), start).flip(1)
    del back
    if s["state"] is not None:
        out["dstate"] = decay[:, 0] * adj[:, 0]
    du = (adj * wide(b)).sum(-1)
    db = (adj * (dt * u)[..., None]).unflatten(2, (g, rep)).sum(3)
    held = torch.cat([state[:, None], h[:, :-1]], 1).mul_(decay).mul_(adj)
    out["da"] = (held * dt[..., None]).sum((0, 1))
    ddt = ((held * a).sum(-1) + du * u) * torch.sigmoid(raw)
    out["dskip"] = (dy * u).sum((0, 1))
    ddt = tokens(ddt)
    out["ddt_bias"] = ddt.flatten(0, -2).sum(0)
    out["ddt"] = ddt.to(type_).view(shape)
    out["du"] = tokens(du * dt + dy * s["skip"]).to(type_).view(shape)
    out["db"], out["dc"] = (tokens(x).to(type_).view(s["b"].shape) for x in (db, dc))
    return out


def _plain_embed(s):
    ids, table = s["ids"].long(), s["table"]
    known = (ids >= 0) & (ids < table.shape[0])
    at = torch.where(known, ids, 0)
    out = {"y": torch.where(known[:, None], table[at].float() * s["scale"], 0.0).to(table.dtype)}
    if s["case"]["do"] == "train":
        dy = torch.where(known[:, None], s["dy"].float() * s["scale"], 0.0)
        out["dtable"] = torch.zeros(table.shape, device="cuda").index_add_(0, at, dy).to(table.dtype)
    return out


def _plain_xent(s):
    h, w, targets = s["h"].float(), s["w"].float(), s["targets"].long()
    counts = (targets >= 0) & (targets < w.shape[0])
    at = torch.where(counts, targets, 0)[:, None]
    z = (h @ w.T) * s["scale"]
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    zero = torch.zeros((), device="cuda")
    out = {"loss": torch.where(counts, (lse - z.gather(1, at))[:, 0], zero), "lse": lse[:, 0]}
    if s["case"]["do"] == "train":
        dloss = torch.where(counts, s["dloss"], zero)[:, None]
        dlse = torch.where(counts, s["dlse"], zero)[:, None] if s["dlse"] is not None else 0.0
        dz = torch.exp(z - lse) * (dloss + dlse)
        dz.scatter_add_(1, at, -dloss)
        dz *= s["scale"]
        out["dh"], out["dw"] = (dz @ w).to(s["h"].dtype), (dz.T @ h).to(s["w"].dtype)
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = 4 if case["type"] == "fp32" else 2
    train = case["do"] == "train"
    if case["op"] == "conv":
        d, k = case["dim"], case["taps"]
        if case["do"] == "step":
            return {"bytes": size * d * case["batch"] * (2 + 2 * (k - 1)), "flops": (2.0 * k + 4) * case["batch"] * d}
        total, held = sum(_lens(case)), (k - 1) * len(_lens(case))
        # x read and y written, the states written (and read); training also reads dy and writes dx
        moved = 2 * total + held * (2 if case["state"] else 1)
        if train:
            moved += 2 * total + (2 * held if case["state"] else 0)
        return {"bytes": size * d * moved, "flops": (2.0 * k + 4) * total * d * (3 if train else 1)}
    if case["op"] == "scan":
        d, n, g = case["dim"], case["states"], case["groups"]
        wide = 4 if case["gate"] else 3  # u, dt and y, and the gate
        if case["do"] == "step":
            b = case["batch"]
            return {"bytes": b * (size * (wide * d + 2 * g * n) + 8 * d * n) + 4 * d * n, "flops": 7.0 * b * d * n}
        total, held = sum(_lens(case)), 4 * d * n * len(_lens(case))
        moved = size * total * (wide * d + 2 * g * n) + held * (2 if case["state"] else 1)
        # the recurrence: a product, an exponential, the state's update and the output's sum for each token, channel and state
        flops = 7.0 * total * d * n
        if train:
            moved += size * total * (wide * d + 2 * g * n) + (2 * held if case["state"] else 0)
            flops += 14.0 * total * d * n
        return {"bytes": moved, "flops": flops}
    if case["op"] == "embed":
        t, d = case["tokens"], case["dim"]
        index = 8 if case["index"] == "i64" else 4
        rows = min(t, case["rows"])
        moved = index * t + size * d * (rows + t)
        if train:
            moved += size * d * (t + case["rows"])
        return {"bytes": moved, "flops": (2.0 if train else 1.0) * t * d}
    m, v, d = case["tokens"], case["vocab"], case["dim"]
    # the logits' product; training: their gradient's two products as well
    return {"bytes": size * (m + v) * d * (2 if train else 1) + 8 * m, "flops": (6.0 if train else 2.0) * m * v * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"conv": _exact_conv, "scan": _exact_scan, "embed": _exact_embed, "xent": _exact_xent}[case["op"]](s)


def _exact_conv(s):
    """One sequence after another, its state in front of it."""
    case = s["case"]
    k, d = case["taps"], case["dim"]
    w, silu = s["w"].double(), case["act"] == "silu"
    bias = s["bias"].double() if s["bias"] is not None else torch.zeros(d, dtype=torch.float64, device="cuda")

    def forward(seq, size):
        p = bias.expand(size, d).clone()
        for j in range(k):
            p += seq[j:j + size] * w[:, j]
        return p, p / (1 + torch.exp(-p)) if silu else p

    if case["do"] == "step":
        state, y = s["state"].double(), []
        for i, slot in enumerate(s["slots"].tolist()):
            seq = torch.cat([state[slot], s["x"][i:i + 1].double()])
            y.append(forward(seq, 1)[1])
            state[slot] = seq[1:]
        return {"y": torch.cat(y), "state": state}
    x, lens = s["x"].reshape(-1, d).double(), _lens(case)
    zero = torch.zeros(k - 1, d, dtype=torch.float64, device="cuda")
    y, final, dx, dinit = [], [], [], []
    dw, dbias = torch.zeros_like(w), torch.zeros_like(bias)
    first = 0
    for i, size in enumerate(lens):
        seq = torch.cat([s["state"][i].double() if s["state"] is not None else zero, x[first:first + size]])
        p, o = forward(seq, size)
        y.append(o)
        final.append(seq[size:])
        if case["do"] == "train":
            dp = s["dy"].reshape(-1, d)[first:first + size].double()
            if silu:
                sig = 1 / (1 + torch.exp(-p))
                dp = dp * (sig + p * sig * (1 - sig))
            dseq = torch.zeros_like(seq)
            for j in range(k):
                dseq[j:j + size] += dp * w[:, j]
                dw[:, j] += (dp * seq[j:j + size]).sum(0)
            dbias += dp.sum(0)
            if s["dstate"] is not None:
                dseq[size:] += s["dstate"][i].double()
            dinit.append(dseq[:k - 1])
            dx.append(dseq[k - 1:])
        first += size
    out = {"y": torch.cat(y).view(s["x"].shape), "final": torch.stack(final)}
    if case["do"] == "train":
        out.update(dx=torch.cat(dx).view(s["x"].shape), dw=dw)
        if s["bias"] is not None:
            out["dbias"] = dbias
        if s["state"] is not None:
            out["dstate"] = torch.stack(dinit)
    return out


def _exact_scan(s):
    """Token by token, one sequence (or, where they are equally long, all of them) at a time."""
    case = s["case"]
    d, n, g = case["dim"], case["states"], case["groups"]
    f64 = dict(dtype=torch.float64, device="cuda")
    group = torch.arange(d, device="cuda") // (d // g)
    a, skip, lift = s["a"].double(), s["skip"].double(), s["dt_bias"].double()

    def steps(raw):
        return torch.where(raw > 0, raw, 0) + torch.log1p(torch.exp(-raw.abs()))

    if case["do"] == "step":
        dt, u = steps(s["dt"].double() + lift), s["u"].double()
        state = s["state"].double()
        at = s["slots"].long()
        state[at] = torch.exp(dt[..., None] * a) * state[at] + (dt * u)[..., None] * s["b"].double()[:, group]
        y = (state[at] * s["c"].double()[:, group]).sum(2) + skip * u
        if s["gate"] is not None:
            z = s["gate"].double()
            y = y * z / (1 + torch.exp(-z))
        return {"y": y, "state": state}

    train = case["do"] == "train"
    parts, first = [], 0
    if case["lens"]:
        for i, size in enumerate(_lens(case)):
            parts.append((slice(i, i + 1), slice(first, first + size)))
            first += size
    else:
        parts.append((slice(0, case["batch"]), None))
    got = []
    sums = {"da": torch.zeros(d, n, **f64), "dskip": torch.zeros(d, **f64), "ddt_bias": torch.zeros(d, **f64)}
    for seqs, span in parts:
        take = lambda x: (x[None, span] if span is not None else x).double()  # noqa: E731
        u, raw, b, c = take(s["u"]), take(s["dt"]) + lift, take(s["b"]), take(s["c"])
        dt = steps(raw)
        count, size = u.shape[:2]
        h = s["state"][seqs].double() if s["state"] is not None else torch.zeros(count, d, n, **f64)
        before = torch.empty(size if train else 0, count, d, n, **f64)
        y = torch.empty(count, size, d, **f64)
        for t in range(size):
            if train:
                before[t] = h
            h = torch.exp(dt[:, t, :, None] * a) * h + (dt[:, t] * u[:, t])[..., None] * b[:, t][:, group]
            y[:, t] = (h * c[:, t][:, group]).sum(2) + skip * u[:, t]
        o = {"final": h.clone()}
        if s["gate"] is not None:
            z = take(s["gate"])
            sig = 1 / (1 + torch.exp(-z))
            o["y"] = y * z * sig
        else:
            o["y"] = y
        if train:
            dy = take(s["dy"])
            if s["gate"] is not None:
                o["dgate"] = dy * y * (sig + z * sig * (1 - sig))
                dy = dy * z * sig
            adj = s["dstate"][seqs].double() if s["dstate"] is not None else torch.zeros(count, d, n, **f64)
            du, ddt = torch.empty_like(u), torch.empty_like(u)
            db, dc = torch.empty_like(b), torch.empty_like(c)
            for t in reversed(range(size)):
                keep = torch.exp(dt[:, t, :, None] * a)
                bt = b[:, t][:, group]
                now = keep * before[t] + (dt[:, t] * u[:, t])[..., None] * bt
                dc[:, t] = (dy[:, t, :, None] * now).view(count, g, d // g, n).sum(2)
                adj = adj + dy[:, t, :, None] * c[:, t][:, group]
                db[:, t] = (adj * (dt[:, t] * u[:, t])[..., None]).view(count, g, d // g, n).sum(2)
                fed = (adj * bt).sum(2)
                du[:, t] = fed * dt[:, t] + skip * dy[:, t]
                moved = adj * keep * before[t]
                ddt[:, t] = fed * u[:, t] + (moved * a).sum(2)
                sums["da"] += (moved * dt[:, t, :, None]).sum(0)
                adj = adj * keep
            ddt = ddt / (1 + torch.exp(-raw))
            sums["dskip"] += (dy * u).sum((0, 1))
            sums["ddt_bias"] += ddt.sum((0, 1))
            o.update(du=du, ddt=ddt, db=db, dc=dc)
            if s["state"] is not None:
                o["dstate"] = adj
        got.append(o)
    like = {"y": "u", "dgate": "u", "du": "u", "ddt": "u", "db": "b", "dc": "c"}
    out = {}
    for name in got[0]:
        if name in like:
            whole = torch.cat([o[name] for o in got], 1) if case["lens"] else got[0][name]
            out[name] = whole.reshape(s[like[name]].shape)
        else:
            out[name] = torch.cat([o[name] for o in got])
    if train:
        out.update(sums)
    return out


def _exact_embed(s):
    """The gradient from sums over the tokens in the order of their numbers."""
    ids, rows = s["ids"].long(), s["case"]["rows"]
    valid = ((ids >= 0) & (ids < rows)).nonzero()[:, 0]
    y = torch.zeros(ids.shape[0], s["case"]["dim"], dtype=torch.float64, device="cuda")
    y[valid] = s["table"].double()[ids[valid]] * s["scale"]
    out = {"y": y}
    if s["case"]["do"] == "train":
        order = valid[ids[valid].argsort(stable=True)]
        total = torch.cat([torch.zeros_like(y[:1]), s["dy"].double()[order].cumsum(0)])
        ends = torch.searchsorted(ids[order], torch.arange(rows + 1, device="cuda"))
        out["dtable"] = (total[ends[1:]] - total[ends[:-1]]) * s["scale"]
    return out


def _exact_xent(s):
    """A block of tokens at a time."""
    w, targets, v = s["w"].double(), s["targets"].tolist(), s["case"]["vocab"]
    m, train = s["case"]["tokens"], s["case"]["do"] == "train"
    f64 = dict(dtype=torch.float64, device="cuda")
    out = {"loss": torch.zeros(m, **f64), "lse": torch.zeros(m, **f64)}
    if train:
        out.update(dh=torch.zeros(s["h"].shape, **f64), dw=torch.zeros(w.shape, **f64))
    step = max(1, min(m, (1 << 27) // v))
    for r0 in range(0, m, step):
        r1 = min(m, r0 + step)
        h = s["h"][r0:r1].double()
        z = torch.mm(h, w.T) * s["scale"]
        lse = torch.logsumexp(z, 1)
        out["lse"][r0:r1] = lse
        rows = [i for i in range(r1 - r0) if 0 <= targets[r0 + i] < v]
        cols = [targets[r0 + i] for i in rows]
        rows, cols = torch.tensor(rows, device="cuda", dtype=torch.long), torch.tensor(cols, device="cuda", dtype=torch.long)
        out["loss"][r0 + rows] = lse[rows] - z[rows, cols]
        if train:
            dloss, dlse = torch.zeros(r1 - r0, **f64), torch.zeros(r1 - r0, **f64)
            dloss[rows] = s["dloss"][r0 + rows].double()
            if s["dlse"] is not None:
                dlse[rows] = s["dlse"][r0 + rows].double()
            dz = torch.softmax(z, 1) * (dloss + dlse)[:, None]
            dz[rows, cols] -= dloss[rows]
            out["dh"][r0:r1] = torch.mm(dz, w) * s["scale"]
            out["dw"] += torch.mm(dz.T, h) * s["scale"]
    return out
