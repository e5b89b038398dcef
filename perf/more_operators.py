"""Cases, plain forms and calls of the gated delta rule, of the verification of
drafted tokens and of the layer norm.

Three operators as a model of delta-rule layers meets them: the norm of the
token rows in front of a layer (``lnorm``), the gated delta rule itself
(``delta``: decode, decode of drafted tokens with every token's state, prefill
and a training step), and the verification that decides how many drafted tokens
stand, and with that which of their states the next step starts from
(``verify``).

Sequence lengths of a case are written as text: ``"8x1024"`` is eight
sequences of 1024 tokens in the fixed layout, ``"5,64,250"`` one packed row of
three sequences, ``"mixed:32:4096:4"`` a packed row of 32 lengths drawn from
[1, 4096] with seed 4.
"""
import math
import random

import torch

own = False

D = 128           # head dimension of the library
CHUNK = 64        # longest block of the plain form
SCALE = 1.0 / math.sqrt(D)
NORM_EPS = 1e-6   # under the root of a query's or key's length
EPS = 1e-5
DEV = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one user's next token through a layer of 32 heads: latency
        dict(name="delta_decode_1", op="delta", mode="decode", lens="1x1", hqk=32, hv=32, slots=4, unit=True),
        # a serving batch's next tokens: bound by the states' way in and out
        dict(name="delta_decode_128", op="delta", mode="decode", lens="128x1", hqk=64, hv=64, slots=160, unit=True),
        # a serving batch's four drafted tokens each, whose states are all kept
        dict(name="delta_draft_32", op="delta", mode="draft", lens="32x5", hqk=16, hv=32, slots=170, unit=True),
        # one long prompt on few heads (a tensor-parallel shard): few rows, a long axis
        dict(name="delta_prefill_long", op="delta", mode="prefill", lens="1x32768", hqk=16, hv=16, slots=2, unit=True),
        # a serving step's mixed prompts, grouped heads
        dict(name="delta_prefill_mixed", op="delta", mode="prefill", lens="mixed:32:4096:4", hqk=16, hv=64, slots=40,
             unit=True),
        # short ragged sequences, as in the tail of a packed batch; keys of unit length as they come
        dict(name="delta_train_ragged", op="delta", mode="train", lens="1,15,16,17,33,100,300", hqk=2, hv=4, unit=False),
        # the packed training batch the library is measured on
        dict(name="delta_train_packed", op="delta", mode="train", lens="packed:8:1024", hqk=96, hv=96, unit=True),
        # grouped heads, fixed layout
        dict(name="delta_train_grouped", op="delta", mode="train", lens="4x4096", hqk=8, hv=32, unit=True),
        # one user's drafts
        dict(name="verify_1", op="verify", n=1, drafts=4, vocab=32000, point=False, ragged=False),
        # a serving batch's drafts, each user with its own number of them
        dict(name="verify_128", op="verify", n=128, drafts=5, vocab=131072, point=False, ragged=True),
        # a decode step's rows
        dict(name="lnorm_infer", op="lnorm", mode="infer", tokens=128, width=4096),
        # a training batch's rows, as wide as the packed batch's 96 heads
        dict(name="lnorm_train", op="lnorm", mode="train", tokens=8192, width=12288),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def _draw_lens(rng, most):
    """Sequence lengths with at most `most` tokens (padding included) in all."""
    kind = rng.choice(("fixed", "packed", "mixed"))
    top = min(most, 32768)
    if kind == "fixed":
        n = _spread(rng, 1, min(16, most))
        return "%dx%d" % (n, _spread(rng, 1, max(1, min(top, most // n))))
    n = _spread(rng, 1, min(32, most))
    top = max(1, min(8192, most // n))
    if kind == "packed":
        return ",".join(str(_spread(rng, 1, top)) for _ in range(min(n, 12)))
    return "mixed:%d:%d:%d" % (n, _spread(rng, 1, top), rng.randrange(1000))


def draw(rng):
    op = rng.choice(("delta", "delta", "delta", "verify", "lnorm"))
    if op == "delta":
        mode = rng.choice(("decode", "draft", "prefill", "train"))
        hqk = _spread(rng, 1, 48)
        hv = hqk * rng.choice((1, 1, 1, 2, 4) if hqk <= 16 else (1,))
        c = dict(op=op, mode=mode, hqk=hqk, hv=hv, unit=rng.random() < 0.7)
        if mode in ("decode", "draft"):
            n = _spread(rng, 1, max(1, min(256, 8192 // hv)))
            tokens = rng.choice((1, 1, 1, 2, 5))
            if mode == "draft":
                n, tokens = max(1, n // 4), rng.choice((2, 3, 5, 8))
            return dict(c, lens="%dx%d" % (n, tokens), slots=n * (tokens if mode == "draft" else 1) + rng.randrange(8))
        lens = _draw_lens(rng, max(64, 400_000 // hv))
        c.update(lens=lens)
        return dict(c, slots=len(_lengths(lens)[0]) + rng.randrange(4)) if mode == "prefill" else c
    if op == "verify":
        vocab = _spread(rng, 17, 200_000)
        drafts = rng.randrange(1, 9)
        n = _spread(rng, 1, max(1, min(256, 100_000_000 // (vocab * (drafts + 1)))))
        return dict(op=op, n=n, drafts=drafts, vocab=vocab, point=rng.random() < 0.3, ragged=rng.random() < 0.5)
    width = 8 * _spread(rng, 4, 2048)
    return dict(op=op, mode=rng.choice(("infer", "train")), tokens=_spread(rng, 1, min(16384, 100_000_000 // width)),
                width=width)


def _lengths(text):
    """(lengths, packed) of a case's lens."""
    if text.startswith("mixed:"):
        _, n, top, seed = text.split(":")
        r = random.Random(int(seed))
        return [r.randint(1, int(top)) for _ in range(int(n))], True
    if text.startswith("packed:"):
        _, n, length = text.split(":")
        return [int(length)] * int(n), True
    if "x" in text:
        n, length = text.split("x")
        return [int(length)] * int(n), False
    return [int(x) for x in text.split(",")], True


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _bf(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "delta":
        lens, packed = _lengths(case["lens"])
        n, hqk, hv = len(lens), case["hqk"], case["hv"]
        b, t = (1, sum(lens)) if packed else (n, lens[0])
        s.update(n=n, longest=max(lens), cu=None, cu_cpu=None)
        if packed:
            s["cu_cpu"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int64)
            s["cu"] = s["cu_cpu"].to(DEV)
        s["q"], s["k"] = _bf(gen, b, t, hqk, D), _bf(gen, b, t, hqk, D)
        if not case["unit"]:  # rows that a norm in front has brought to unit length
            s["q"], s["k"] = ((x.float() / x.float().square().sum(-1, keepdim=True).sqrt()).bfloat16() for x in (s["q"], s["k"]))
        s["v"] = _bf(gen, b, t, hv, D)
        # decays as a layer starts out with: rates 1 to 16 over its heads, steps of 0.001 to 0.1, moved by the token
        rate = 1 + 15 * torch.rand(hv, generator=gen, device=DEV)
        step = 0.001 * 100.0 ** torch.rand(hv, generator=gen, device=DEV)
        shift = torch.log(torch.expm1(step))
        s["g"] = (-rate * torch.nn.functional.softplus(_randn(gen, b, t, hv) + shift)).bfloat16()
        s["beta"] = torch.sigmoid(_randn(gen, b, t, hv)).bfloat16()
        if case["mode"] == "train":
            s["state"] = _randn(gen, n, hv, D, D) * 0.1
            s["do"] = _bf(gen, b, t, hv, D)
            s["dstate"] = _randn(gen, n, hv, D, D) * 0.1
        else:
            s["pool"] = _randn(gen, case["slots"], hv, D, D) * 0.1
            each = lens[0] if case["mode"] == "draft" else 1
            slots = torch.randperm(case["slots"], generator=torch.Generator().manual_seed(seed))[:n * each]
            s["slot_cpu"] = slots.to(torch.int32).reshape((n, each) if case["mode"] == "draft" else (n,)).contiguous()
            s["slot"] = s["slot_cpu"].to(DEV)
            if case["mode"] == "draft":
                s["accepted"] = torch.randint(1, each + 1, (n,), generator=gen, device=DEV, dtype=torch.int32)
        return s
    if case["op"] == "verify":
        n, m, v = case["n"], case["drafts"], case["vocab"]
        logits = 3 * _randn(gen, n, m + 1, v)
        s["target"] = torch.softmax(logits, -1)
        if case["point"]:  # drafts that are given as they are, such as found in the text before
            s["draft"] = None
            drawn = s["target"][:, :m]
        else:
            s["draft"] = drawn = torch.softmax(0.9 * logits[:, :m] + 0.3 * _randn(gen, n, m, v), -1)
        race = -torch.log(torch.rand(n, m, v, generator=gen, device=DEV).clamp_min(1e-30))
        s["tokens"] = (drawn / race).argmax(-1).to(torch.int32)
        s["lens"] = torch.randint(0, m + 1, (n,), generator=gen, device=DEV, dtype=torch.int32) if case["ragged"] else None
        s["uniform"] = torch.rand(n, m + 1, generator=gen, device=DEV)
        return s
    t, w = case["tokens"], case["width"]
    s["x"] = (_randn(gen, t, w) + 0.5 * _randn(gen, t, 1)).bfloat16()
    s["w"], s["b"] = 1 + 0.1 * _randn(gen, w), 0.1 * _randn(gen, w)
    if case["mode"] == "train":
        s["dy"] = _bf(gen, t, w)
    return s


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------
def _own(s):
    import gated_delta_rule_32_amd as kda
    c = s["case"]
    if c["op"] == "delta":
        a = (s["q"], s["k"], s["v"], s["g"], s["beta"])
        if c["mode"] == "train":
            o, fs, ctx = kda.gated_delta_rule_training_forward(*a, s["state"], cu_seqlens=s["cu"], cu_seqlens_cpu=s["cu_cpu"],
                                                               use_qk_l2norm=c["unit"])
            return (o, fs) + tuple(kda.gated_delta_rule_training_backward(ctx, s["do"], s["dstate"]))
        more = dict(num_spec_tokens=s["longest"] - 1, num_accepted_tokens=s["accepted"]) if c["mode"] == "draft" else {}
        return kda.gated_delta_rule(*a, s["pool"], cu_seqlens=s["cu"], cu_seqlens_cpu=s["cu_cpu"], ssm_state_indices=s["slot"],
                                    ssm_state_indices_cpu=s["slot_cpu"], use_qk_l2norm=c["unit"], **more)
    if c["op"] == "verify":
        return kda.verify_drafts(s["tokens"], s["target"], s["uniform"], s["draft"], s["lens"])
    y = kda.layer_norm_forward(s["x"], s["w"], s["b"], eps=EPS)
    if c["mode"] == "infer":
        return y
    return (y,) + tuple(kda.layer_norm_backward(s["dy"], s["x"], s["w"], eps=EPS))


def run(state):
    if own:
        return _own(state)
    return {"delta": _plain_delta, "verify": _plain_verify, "lnorm": _plain_lnorm}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# plain forms, in 32 bits
# --------------------------------------------------------------------------
def _rows(s):
    """[N, L'] token rows of every sequence, padded to a whole number of
    blocks, and which of them hold a token."""
    n, b_t = s["n"], s["q"].shape[1]
    block = min(CHUNK, s["longest"])
    width = -(-s["longest"] // block) * block
    start = s["cu"][:-1] if s["cu"] is not None else torch.arange(n, device=DEV) * b_t
    length = s["cu"].diff() if s["cu"] is not None else torch.full((n,), b_t, device=DEV)
    at = torch.arange(width, device=DEV)
    there = at < length[:, None]
    return torch.where(there, start[:, None] + at, 0), there, block


def _lay(x, heads, rows, there):
    """[B, T, H, ...] tokens as FP32 [N, heads, L', ...], zero where no token is."""
    x = x.reshape(-1, *x.shape[2:])[rows].float()
    x = x * there.reshape(there.shape + (1,) * (x.dim() - 2))
    return x.repeat_interleave(heads // x.shape[2], 2).transpose(1, 2)


def _back(y, rows, there, like):
    """The reverse of _lay, rounded."""
    out = torch.zeros((like.shape[0] * like.shape[1], y.shape[1], *y.shape[3:]), device=DEV)
    out[rows[there]] = y.transpose(1, 2)[there]
    return out.reshape(like.shape[0], like.shape[1], *out.shape[1:]).bfloat16()


def _unit(x, on):
    """Rows at unit length, and one over the length that they had."""
    r = torch.rsqrt(x.square().sum(-1, keepdim=True) + NORM_EPS) if on else torch.ones_like(x[..., :1])
    return x * r, r


def _unit_back(d, hat, r, on):
    return r * (d - hat * (d * hat).sum(-1, keepdim=True)) if on else d


def _t(x):
    return x.transpose(-1, -2)


def _plain_tokens(s):
    """The recurrence itself, for calls of a few tokens."""
    c, hv = s["case"], s["case"]["hv"]
    draft = c["mode"] == "draft"
    wide = lambda x: x.float().repeat_interleave(hv // x.shape[2], 2)  # noqa: E731
    q, k, v = _unit(wide(s["q"]), c["unit"])[0], _unit(wide(s["k"]), c["unit"])[0], s["v"].float()
    alpha, beta = torch.exp(s["g"].float()), s["beta"].float()
    slot = s["slot"].long()
    first = slot.gather(1, s["accepted"].long()[:, None] - 1)[:, 0] if draft else slot
    x = s["pool"][first]
    o = torch.empty_like(s["v"])
    for t in range(s["longest"]):
        x = x * alpha[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (x * k[:, t, :, None]).sum(-1))
        x = x + u[..., None] * k[:, t, :, None]
        o[:, t] = (SCALE * (x * q[:, t, :, None]).sum(-1)).bfloat16()
        if draft:
            s["pool"][slot[:, t]] = x
    if not draft:
        s["pool"][slot] = x
    return o, s["pool"]


def _plain_delta(s):
    c, hv = s["case"], s["case"]["hv"]
    if c["mode"] in ("decode", "draft"):
        return _plain_tokens(s)
    train = c["mode"] == "train"
    rows, there, block = _rows(s)
    n, blocks = s["n"], rows.shape[1] // block
    chunks = lambda x: x.reshape(n, hv, blocks, block, *x.shape[3:])  # noqa: E731
    lay = lambda x: chunks(_lay(x, hv, rows, there))  # noqa: E731
    (q, rq), (k, rk), v = _unit(lay(s["q"]), c["unit"]), _unit(lay(s["k"]), c["unit"]), lay(s["v"])
    beta = lay(s["beta"])[..., None]
    # decays: sums of logarithms in 64 bits, their differences rounded once
    acc = lay(s["g"]).double().cumsum(-1)
    low = torch.ones(block, block, device=DEV, dtype=torch.bool).tril()
    gap = torch.where(low, acc[..., :, None] - acc[..., None, :], -torch.inf).exp().float()   # e^{G_i - G_j}, j <= i
    since = acc.exp().float()[..., None]                     # e^{G_i}
    left = (acc[..., -1:] - acc).exp().float()[..., None]    # e^{G_last - G_i}
    whole = acc[..., -1].exp().float()[..., None, None]      # of the block
    kk = (k @ _t(k)) * gap
    kk = kk - torch.diag_embed(kk.diagonal(dim1=-2, dim2=-1))
    # inv = (1 + kk diag(beta))^-1, row after row
    mat = kk * _t(beta)
    inv = torch.eye(block, device=DEV).expand_as(mat).clone()
    for i in range(1, block):
        inv[..., i, :i] = -(mat[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    qk = SCALE * (q @ _t(k)) * gap
    base, reach = inv @ v, inv @ (k * since)
    state = _t(s["state"] if train else s["pool"][s["slot"].long()])   # [k][v]
    starts, ws = [], []
    for i in range(blocks):
        starts.append(state)
        ws.append(base[:, :, i] - reach[:, :, i] @ state)
        state = whole[:, :, i] * state + _t(k[:, :, i] * left[:, :, i] * beta[:, :, i]) @ ws[-1]
    w, start = torch.stack(ws, 2), torch.stack(starts, 2)
    u = beta * w
    o = SCALE * since * (q @ start) + qk @ u
    flat = lambda x: x.reshape(n, hv, blocks * block, *x.shape[4:])  # noqa: E731
    back = lambda x: _back(flat(x), rows, there, s["q"])  # noqa: E731
    final = _t(state).contiguous()
    if not train:
        s["pool"][s["slot"].long()] = final
        return back(o), s["pool"]
    # backward in time: y, the adjoint of u, and the state's adjoint behind every block
    do = lay(s["do"])
    beside = _t(qk) @ do
    adj = _t(s["dstate"])
    # (1 + kk^T diag(beta))^-1 = 1 - (diag(beta) kk inverted)^T, from inv without dividing by beta
    turn = torch.eye(block, device=DEV) - _t(inv @ kk) @ torch.diag_embed(beta[..., 0])
    ends, ys = [], []
    for i in reversed(range(blocks)):
        ends.append(adj)
        ys.append(turn[:, :, i] @ (beside[:, :, i] + left[:, :, i] * (k[:, :, i] @ adj)))
        adj = whole[:, :, i] * adj + _t(SCALE * since[:, :, i] * q[:, :, i]) @ do[:, :, i] \
            - _t(since[:, :, i] * k[:, :, i]) @ (beta[:, :, i] * ys[-1])
    y, end = torch.stack(ys[::-1], 2), torch.stack(ends[::-1], 2)
    dw = beta * y
    e, f = SCALE * (do @ _t(u)) * gap, (dw @ _t(u)) * gap.tril(-1)
    dq_s, dk_s, dk_e = SCALE * since * (do @ _t(start)), -since * (dw @ _t(start)), left * (u @ _t(end))
    dq = dq_s + e @ k
    dk = dk_s + dk_e + _t(e) @ q - _t(f) @ k - f @ k
    dbeta = (y * w).sum(-1)
    # a decay acts on all that passes its token: what stands before against what comes from it on
    h = (e * (q @ _t(k)) - f * (k @ _t(k))).tril(-1)
    passes = (h.sum(-2) - h.sum(-1)).cumsum(-1) - (h.sum(-2) - h.sum(-1))
    here = (q * dq_s).sum(-1) + (k * dk_s).sum(-1)
    on = (k * dk_e).sum(-1)
    dg = (whole * end * start).sum((-1, -2))[..., None] + on.cumsum(-1) - on + here.flip(-1).cumsum(-1).flip(-1) + passes
    dq, dk = _unit_back(dq, q, rq, c["unit"]), _unit_back(dk, k, rk, c["unit"])
    shared = lambda x: x.unflatten(1, (-1, hv // c["hqk"])).sum(2)  # noqa: E731
    fold = lambda x: _back(shared(flat(x)), rows, there, s["q"])  # noqa: E731
    return back(o), final, fold(dq), fold(dk), back(dw), back(dg), back(dbeta), _t(adj).contiguous()


def _plain_verify(s):
    p, q, x = s["target"], s["draft"], s["tokens"].long()
    n, m = x.shape
    draws = s["uniform"].double()
    lens = s["lens"].long() if s["lens"] is not None else torch.full((n,), m, device=DEV)
    px = p[:, :m].gather(2, x[..., None])[..., 0].double()
    qx = q.gather(2, x[..., None])[..., 0].double() if q is not None else 1.0
    place = torch.arange(m + 1, device=DEV)
    fine = (draws[:, :m] * qx < px) & (place[:m] < lens[:, None])
    stand = fine.long().cumprod(1).sum(1)
    # the row to draw from: what the target has more than the draft, or the target's own behind the last draft
    pick = torch.arange(n, device=DEV)
    row = p[pick, stand].double()
    at = stand.clamp(max=m - 1)
    took = q[pick, at].double() if q is not None else (torch.arange(row.shape[1], device=DEV) == x[pick, at][:, None]).double()
    more = (row - took).clamp(min=0)
    more = torch.where((stand < lens)[:, None] & (more.sum(1, keepdim=True) > 0), more, row)
    run_ = more.cumsum(1)
    past = (run_ > draws[:, m:].clamp(min=0) * run_[:, -1:]) & (more > 0)
    last = row.shape[1] - 1 - (more > 0).flip(1).long().argmax(1)
    drawn = torch.where(past.any(1), past.long().argmax(1), last)
    tokens = torch.cat((x, x[:, :1]), 1)
    tokens = torch.where(place == stand[:, None], drawn[:, None], torch.where(place < stand[:, None], tokens, -1))
    return tokens.to(torch.int32), (stand + 1).to(torch.int32)


def _plain_lnorm(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    r = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
    hat = (x - mean) * r
    y = (hat * s["w"] + s["b"]).bfloat16()
    if s["case"]["mode"] == "infer":
        return y
    dy = s["dy"].float()
    d = dy * s["w"]
    dx = r * (d - d.mean(-1, keepdim=True) - hat * (d * hat).mean(-1, keepdim=True))
    return y, dx.bfloat16(), (dy * hat).sum(0), dy.sum(0)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "delta":
        lens, _ = _lengths(case["lens"])
        t, hqk, hv = sum(lens), case["hqk"], case["hv"]
        states = len(lens) * hv * D * D * 4
        gates = t * hv * 2 * 2
        # S k, the state's update and S q; the backward adds the states again, their adjoint and four read-outs
        if case["mode"] == "train":
            return {"bytes": t * (4 * hqk + 4 * hv) * D * 2 + 2 * gates + 4 * states, "flops": 22 * D * D * t * hv}
        out = lens[0] if case["mode"] == "draft" else 1
        return {"bytes": t * (2 * hqk + 2 * hv) * D * 2 + gates + (1 + out) * states, "flops": 6 * D * D * t * hv}
    if case["op"] == "verify":
        row = case["vocab"] * 4 * (1 if case["point"] else 2)
        return {"bytes": case["n"] * (row + case["drafts"] * 24), "flops": case["n"] * 4 * case["vocab"]}
    train = case["mode"] == "train"
    return {"bytes": case["tokens"] * case["width"] * 2 * (4 if train else 2) + case["width"] * (16 if train else 8),
            "flops": case["tokens"] * case["width"] * (18 if train else 7)}


# --------------------------------------------------------------------------
# the operators' definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return None  # whole numbers: nothing that a rounding moves
    return (_exact_delta if case["op"] == "delta" else _exact_lnorm)(s)


def _exact_delta(s):
    """The recurrence, token by token, S[v][k]: S <- e^g S, S <- S + beta (v -
    S k) k^T, o = S q / sqrt(D); and its adjoint, from the last token to the
    first, with the states kept at every 64th token and run again between."""
    c, n, hv = s["case"], s["n"], s["case"]["hv"]
    train, draft = c["mode"] == "train", c["mode"] == "draft"
    b, t = s["q"].shape[:2]
    lens = s["cu_cpu"].diff().tolist() if s["cu_cpu"] is not None else [t] * n
    starts = s["cu_cpu"][:-1].tolist() if s["cu_cpu"] is not None else [i * t for i in range(n)]
    # longest first, so that the sequences that still run are a leading slice
    order = sorted(range(n), key=lambda i: -lens[i])
    first = torch.tensor([starts[i] for i in order], device=DEV)
    size = torch.tensor([lens[i] for i in order])
    running = [(size > i).sum().item() for i in range(int(size.max()))]
    pick = torch.tensor(order, device=DEV)
    flat = {x: s[x].reshape(b * t, *s[x].shape[2:]) for x in ("q", "k", "v", "g", "beta", "do") if x in s}

    def token(name, at):
        return flat[name][at].double().repeat_interleave(hv // flat[name].shape[1], 1)

    def length(x):
        return (x.square().sum(-1, keepdim=True) + NORM_EPS).sqrt() if c["unit"] else torch.ones_like(x[..., :1])

    def inputs(i):
        at = first[:running[i]] + i
        q, k = token("q", at), token("k", at)
        nq, nk = length(q), length(k)
        return at, q / nq, k / nk, nq, nk, token("v", at), token("g", at).exp()[..., None, None], token("beta", at)[..., None]

    def dot(a, x):  # a row of x against every row of a
        return (a @ x[..., None])[..., 0]

    def step(live, a, k, v, beta):
        live.mul_(a)
        w = v - dot(live, k)
        live.add_((beta * w)[..., None] * k[:, :, None])
        return w

    if train:
        state = s["state"][pick].double()
    elif draft:
        state = s["pool"][s["slot"].long().gather(1, s["accepted"].long()[:, None] - 1)[:, 0]][pick].double()
    else:
        state = s["pool"][s["slot"].long()[pick]].double()
    pool = None if train else s["pool"].double()
    o = torch.zeros(b * t, hv, D, device=DEV, dtype=torch.float64)
    kept = []
    for i, m in enumerate(running):
        if train and i % 64 == 0:
            kept.append(state[:m].clone())
        at, q, k, _, _, v, a, beta = inputs(i)
        step(state[:m], a, k, v, beta)
        o[at] = dot(state[:m], q) * SCALE
        if draft:
            pool[s["slot"].long()[pick, i]] = state
    shape = lambda x: x.reshape(b, t, *x.shape[1:])  # noqa: E731
    if not train:
        if not draft:
            pool[s["slot"].long()[pick]] = state
        return shape(o), pool
    final = torch.empty_like(state)
    final[pick] = state
    dq, dk, dv = (torch.zeros_like(o) for _ in range(3))
    dg, dbeta = (torch.zeros(b * t, hv, device=DEV, dtype=torch.float64) for _ in range(2))
    adj = s["dstate"][pick].double()
    for block in reversed(range(len(kept))):
        tokens = range(64 * block, min(64 * block + 64, len(running)))
        state, before = kept[block], []
        for i in tokens:  # the states in front of every token
            state = state[:running[i]]
            before.append(state.clone())
            _, _, k, _, _, v, a, beta = inputs(i)
            step(state, a, k, v, beta)
        for i in reversed(tokens):
            at, q, k, nq, nk, v, a, beta = inputs(i)
            live, x = adj[:running[i]], before.pop()
            x.mul_(a)                          # decayed
            w = v - dot(x, k)
            do = token("do", at) * SCALE
            live.add_(do[..., None] * q[:, :, None])
            du = dot(live, k)                  # adjoint of beta w
            gq = dot(_t(x), do) + (do * beta * w).sum(-1, keepdim=True) * k
            gk = dot(_t(live), beta * w) - dot(_t(x), beta * du)
            dv[at], dbeta[at] = beta * du, (du * w).sum(-1)
            live.sub_((beta * du)[..., None] * k[:, :, None])
            dg[at] = (live * x).sum((-1, -2))
            live.mul_(a)
            for out, d, hat, size_ in ((dq, gq, q, nq), (dk, gk, k, nk)):
                out[at] = (d - hat * (d * hat).sum(-1, keepdim=True)) / size_ if c["unit"] else d
    dinit = torch.empty_like(adj)
    dinit[pick] = adj
    shared = lambda x: x.unflatten(1, (-1, hv // c["hqk"])).sum(2)  # noqa: E731
    return shape(o), final, shape(shared(dq)), shape(shared(dk)), shape(dv), shape(dg), shape(dbeta), dinit


def _exact_lnorm(s):
    x, w = s["x"].double(), s["w"].double()
    mean = x.mean(-1, keepdim=True)
    norm = ((x * x).mean(-1, keepdim=True) - mean * mean + EPS).sqrt()
    y = (x - mean) / norm * w + s["b"].double()
    if s["case"]["mode"] == "infer":
        return y
    dy = s["dy"].double()
    u = dy * w / norm
    hat = (x - mean) / norm
    return y, u - u.mean(-1, keepdim=True) - hat * (u * hat).mean(-1, keepdim=True), (dy * hat).sum(0), dy.sum(0)
