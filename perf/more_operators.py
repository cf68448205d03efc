"""What a recurrent text model needs beside its mixing operators, as measured
cases: the gated scan (a layer), the clipping of a training step's gradients by
their global norm, and for answering with beams the selection over beams and
vocabulary and the reordering of the carried states.

Each case is one pass of one operator.  ``run`` computes it in the plain form
(elementary torch operations) while ``own`` is false and through the package's
entry points while it is true; ``exact`` evaluates the definition in 64 bits.
Windows are time first ([T, B, channels]), as everywhere in the package.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases

def _scan(name, op, T, B, D, dtype, input_gate, z, ragged, layout):
    return {"name": name, "op": op, "T": T, "B": B, "D": D, "dtype": dtype,
            "input_gate": input_gate, "z": z, "ragged": ragged, "layout": layout}


def _clip(name, tensors, total, dtype, factor, odd):
    """`total` elements in `tensors` gradients, the i-th about 1 / (i + 1) of the
    first; factor: the limit, as a part of the norm the inputs are drawn with."""
    return {"name": name, "op": "clip", "tensors": tensors, "total": total, "dtype": dtype,
            "factor": factor, "odd": odd}


def _select(name, B, K, V, dtype, finished, pad):
    return {"name": name, "op": "beam_select", "B": B, "K": K, "V": V, "dtype": dtype,
            "finished": finished, "pad": pad}


def _reorder(name, B, K, D, N, W, nodes, dtype):
    return {"name": name, "op": "beam_reorder", "B": B, "K": K, "D": D, "N": N, "W": W,
            "nodes": nodes, "dtype": dtype}


def listed():
    return [
        # training on the FlyGPT window (64 steps, batch 32) over its 256 input channels
        _scan("gated_train_window", "gated_train", 64, 32, 256, "fp32", False, False, False, "time"),
        # training on long texts, all gates slices of one projection
        _scan("gated_train_text", "gated_train", 2048, 8, 2048, "bf16", True, True, False, "proj"),
        # training on texts of unequal length (none to all of the window), odd channels
        _scan("gated_train_ragged", "gated_train", 777, 5, 1001, "fp16", True, False, True, "batch"),
        # one long prompt read before answering: a single row
        _scan("gated_prompt_long", "gated_prompt", 16384, 1, 2048, "bf16", True, True, False, "proj"),
        # answering, one token for one text: the smallest call of the scan
        _scan("gated_token_one", "gated_token", 1, 1, 256, "bf16", True, True, False, "proj"),
        # the gradients of a model around the FlyGPT graph: few tensors, half a million edges
        _clip("clip_flygpt", 14, 700_000, "fp32", 0.25, False),
        # the gradients of the whole-connectome graph's model, fp32
        _clip("clip_connectome", 14, 26_000_000, "fp32", 0.25, False),
        # many 16-bit gradients of odd sizes, within the limit: copied unscaled
        _clip("clip_many", 60, 60_000_001, "bf16", 4.0, True),
        # the smallest selection: one text, the text example's alphabet
        _select("beam_select_one", 1, 4, 28, "fp32", False, 0),
        # many texts over a whole vocabulary, some beams finished, rows of a padded projection
        _select("beam_select_many", 64, 8, 50_021, "bf16", True, 27),
        # the states of one text's beams: convolution, scan, gated scan, nodes
        _reorder("beam_reorder_one", 1, 4, 256, 16, 4, 5000, "bf16"),
        # the states of many texts' beams
        _reorder("beam_reorder_many", 64, 8, 2048, 16, 4, 5000, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_train", "gated_train", "gated_prompt", "gated_prompt", "gated_token",
                     "clip", "clip", "beam_select", "beam_select", "beam_reorder"])
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    one, two = rng.random() < 0.5, rng.random() < 0.5
    if op == "clip":
        return _clip("", _log_int(rng, 1, 60), _log_int(rng, 10_000, 40_000_000), dtype,
                     rng.choice([0.25, 0.5, 4.0]), one)
    if op == "beam_select":
        K, V = _log_int(rng, 1, 32), _log_int(rng, 28, 200_000)
        B = _log_int(rng, 1, max(1, min(64, 64 * 8 * 50_021 // (2 * K * V))))
        return _select("", B, K, V, dtype, one, rng.choice([0, 0, rng.randint(1, 64)]))
    if op == "beam_reorder":
        K, D, N = _log_int(rng, 1, 32), _log_int(rng, 16, 2048), rng.randint(1, 16)
        B = _log_int(rng, 1, max(1, min(64, 64 * 8 * 2048 // (K * D))))
        return _reorder("", B, K, D, N, rng.randint(2, 4), _log_int(rng, 28, 5000), dtype)
    ragged, layout = rng.random() < 0.4, rng.choice(["time", "batch", "proj"])
    D = _log_int(rng, 64, 2048)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    if op == "gated_token":
        return _scan("", op, 1, _log_int(rng, 1, 256), D, dtype, one, two, False, layout)
    T = _log_int(rng, 33, 16384 if op == "gated_prompt" else 2048)
    # the listed cases' largest sizes bound a draw's positions
    B = _log_int(rng, 1, max(1, min(64, 1024 * 8 * 2048 // (T * D))))
    return _scan("", op, T, B, D, dtype, one, two, ragged, layout)


def _lengths(case):
    """Ragged batches hold texts of evenly spread lengths, from none to all of T."""
    T, B = case["T"], case["B"]
    if not case.get("ragged"):
        return [T] * B
    return [T * b // (B - 1) for b in range(B)] if B > 1 else [T // 2]


def _sizes(case):
    """Elements of each gradient of a clipping case."""
    n = case["tensors"]
    share = case["total"] / sum(1 / (i + 1) for i in range(n))
    sizes = [max(1, int(share / (i + 1))) for i in range(n)]
    return [s | 1 for s in sizes] if case["odd"] else sizes


def _done(case):
    """Which beams of a selection are finished: every fifth, but a text's first."""
    B, K = case["B"], case["K"]
    return [[case["finished"] and k > 0 and (b + k) % 5 == 0 for k in range(K)] for b in range(B)]


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * n * e + 4, "flops": 3 * n}
    if case["op"] == "beam_select":
        B, K, V = case["B"], case["K"], case["V"]
        # a finished beam's logits need not be read
        live = sum(not f for row in _done(case) for f in row)
        return {"bytes": live * V * e + B * K * (2 * (4 + 1) + 16), "flops": 4 * live * V}
    if case["op"] == "beam_reorder":
        rows = case["B"] * case["K"]
        row = (case["W"] - 1) * case["D"] * e + 4 * (case["D"] * (case["N"] + 1) + case["nodes"])
        return {"bytes": 2 * rows * row + 8 * rows, "flops": 0}
    T, B, D = case["T"], case["B"], case["D"]
    rows = sum(_lengths(case))
    x, out = rows * D * e, T * B * D * e   # outputs are written over the whole window
    gates = 1 + int(case["input_gate"]) + int(case["z"])
    state, par = B * D * 4, 2 * D * 4
    bytes_ = (1 + gates) * x + out + 2 * state + par
    flops = rows * D * (4 + 4 * gates)
    if case["op"] == "gated_train":        # the forward, then the backward with its upstream gradient
        bytes_ += (2 + gates) * x + (1 + gates) * out + 2 * state + 2 * par
        flops += rows * D * (10 + 12 * gates)
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------- the inputs

def _gates(g, case, dtype):
    """x and its gates [T, B, D] in the case's storage: time or batch outermost,
    or slices of one projection's output."""
    T, B, D = case["T"], case["B"], case["D"]
    n = 2 + int(case["input_gate"]) + int(case["z"])

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    if case["layout"] == "proj":
        parts = list(rand(T, B, n * D).split(D, dim=-1))
    elif case["layout"] == "batch":
        parts = [rand(B, T, D).transpose(0, 1) for _ in range(n)]
    else:
        parts = [rand(T, B, D) for _ in range(n)]
    x, f = parts[:2]
    i = parts[2] if case["input_gate"] else None
    return x, f, i, parts[-1] if case["z"] else None


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    st = {"case": case}
    if case["op"] == "clip":
        # gradients of unlike scales, as layers have them
        sizes = _sizes(case)
        scales = torch.exp(2 * randn(len(sizes))).tolist()
        st["grads"] = [(s * 1e-3 * randn(n)).to(dtype) for s, n in zip(scales, sizes)]
        st["outs"] = [torch.empty_like(t) for t in st["grads"]]
        drawn = math.sqrt(sum((1e-3 * s) ** 2 * n for s, n in zip(scales, sizes)))
        st["max_norm"] = case["factor"] * drawn
        return st
    if case["op"] == "beam_select":
        B, K, V = case["B"], case["K"], case["V"]
        # a padded projection's rows, of which the vocabulary is a slice
        st["logits"] = (3 * randn(B, K, V + case["pad"])).to(dtype)[:, :, :V]
        st["scores"] = -20 * rand(B, K)
        st["finished"], st["eos"] = None, None
        if case["finished"]:
            st["finished"] = torch.tensor(_done(case), device="cuda")
            st["eos"] = 2
        return st
    if case["op"] == "beam_reorder":
        B, K, D = case["B"], case["K"], case["D"]
        rows = B * K
        conv = randn(case["W"] - 1, rows, D).to(dtype)      # steps first: rows are its second axis
        states = [conv.transpose(0, 1), randn(rows, D, case["N"]), randn(rows, D),
                  randn(rows, case["nodes"])]
        st["states"] = states
        st["outs"] = [torch.empty_like(conv).transpose(0, 1)] + \
            [torch.empty_like(t) for t in states[1:]]
        # a few beams carry most of what goes on
        st["parents"] = (rand(B, K).square() * K).long()
        return st
    T, B, D = case["T"], case["B"], case["D"]
    st["lengths"] = None
    if case["ragged"]:
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    st["x"], st["f"], st["i"], st["z"] = _gates(g, case, dtype)
    keep = 0.9 + 0.099 * rand(D)           # what such layers keep of a state when they start
    st["f_bias"] = torch.log(keep / (1 - keep))
    st["i_bias"] = 0.5 * randn(D) if case["input_gate"] else None
    st["state0"] = 0.5 * randn(B, D)
    if case["op"] == "gated_train":
        st["grad_out"] = randn(T, B, D).to(dtype)
        st["grad_state"] = randn(B, D)
    if case["op"] == "gated_token":
        st["new_state"] = torch.empty_like(st["state0"])
    return st


# ----------------------------------------------------------- the plain forms

def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _masked(x, valid, other=0.0):
    return x if valid is None else torch.where(valid, x, other)


def _linear_scan(a, u):
    """All h_t = a_t h_{t-1} + u_t (h_{-1} = 0) by doubling the steps that a pair spans."""
    a, u, span = a.clone(), u.clone(), 1
    while span < a.shape[0]:
        u[span:] += a[span:] * u[:-span]
        a[span:] = a[span:] * a[:-span]
        span *= 2
    return u


def _plain_gated(st, train):
    case, dtype = st["case"], st["x"].dtype
    T = case["T"]
    valid = None
    if st["lengths"] is not None:
        valid = (torch.arange(T, device="cuda")[:, None] < st["lengths"][None, :]).unsqueeze(-1)
    x = _masked(st["x"].float(), valid)
    # a gate that is almost 1 is held as what is missing from it
    leave = _masked(_sigmoid(-(_masked(st["f"].float(), valid) + st["f_bias"])), valid)
    keep = 1 - leave
    if st["i"] is None:
        take = leave
    else:
        take = _masked(_sigmoid(_masked(st["i"].float(), valid) + st["i_bias"]), valid)
    u = take * x
    u[0] += keep[0] * st["state0"]
    h = _linear_scan(keep, u)
    gate = None
    if st["z"] is not None:
        z = _masked(st["z"].float(), valid)
        sz = _sigmoid(z)
        gate = z * sz
    out = _masked(h if gate is None else h * gate, valid).to(dtype)
    state = h[-1].clone()
    if not train:
        return [out, state]
    go = _masked(st["grad_out"].float(), valid)
    y = go if gate is None else go * gate
    y = y.flip(0)
    y[0] += st["grad_state"]
    after = torch.cat([torch.ones_like(keep[:1]), keep[1:].flip(0)])
    gh = _linear_scan(after, y).flip(0)
    before = torch.cat([st["state0"].unsqueeze(0), h[:-1]])
    gx = (gh * take).to(dtype)
    if st["i"] is None:
        gf = gh * (before - x) * keep * leave
    else:
        gf = gh * before * keep * leave
    grads = [gx, gf.to(dtype), gf.double().sum((0, 1)).float(), keep[0] * gh[0]]
    if st["i"] is not None:
        gi = gh * x * take * (1 - take)
        grads += [gi.to(dtype), gi.double().sum((0, 1)).float()]
    if gate is not None:
        grads.append((go * h * sz * (1 + z * (1 - sz))).to(dtype))
    return [out, state] + grads


def _plain_clip(st):
    square = sum(t.double().square().sum() for t in st["grads"])
    norm = square.sqrt()
    scale = torch.where(norm > st["max_norm"], st["max_norm"] / norm, torch.ones_like(norm)).float()
    return [norm.float().view(1)] + [(t.float() * scale).to(t.dtype) for t in st["grads"]]


def _plain_select(st):
    """In 64 bits: which of two candidates is the better one is a border."""
    case, logits = st["case"], st["logits"]
    B, K, V = case["B"], case["K"], case["V"]
    x = logits.double()
    top = x.amax(-1, keepdim=True)
    total = torch.exp(x - top).sum(-1, keepdim=True)
    x = st["scores"].double().unsqueeze(-1) + ((x - top) - torch.log(total))
    if st["finished"] is not None:         # goes on with the end token alone, at its score
        stays = torch.full_like(x, -math.inf)
        stays[:, :, st["eos"]] = st["scores"].double()
        x = torch.where(st["finished"].unsqueeze(-1), stays, x)
    x = x.view(B, K * V)
    free = torch.ones_like(x, dtype=torch.bool)
    scores, flat = [], []
    for _ in range(K):                     # the best left, the first of those that are equal
        best = torch.where(free, x, -math.inf).amax(-1, keepdim=True)
        at = ((x == best) & free).to(torch.uint8).argmax(-1, keepdim=True)
        free.scatter_(1, at, False)
        scores.append(best)
        flat.append(at)
    scores, flat = torch.cat(scores, 1).float(), torch.cat(flat, 1)
    parents, tokens = flat // V, flat % V
    if st["finished"] is None:
        return [scores, parents, tokens]
    return [scores, parents, tokens, st["finished"].gather(1, parents) | (tokens == st["eos"])]


def _plain_reorder(st):
    B, K = st["parents"].shape
    rows = (st["parents"] + K * torch.arange(B, device="cuda").unsqueeze(1)).view(-1)
    return [t[rows] for t in st["states"]]


def _own(st):
    import sparse_graph_recurrent_amd as sgr

    case = st["case"]
    op = case["op"]
    if op == "clip":
        norm, outs = sgr.clip_grad_norm(st["grads"], st["max_norm"], out=st["outs"])
        return [norm] + list(outs)
    if op == "beam_select":
        got = sgr.beam_select(st["logits"], st["scores"], st["finished"], st["eos"])
        return list(got) if st["finished"] is not None else list(got[:3])
    if op == "beam_reorder":
        return list(sgr.beam_reorder(st["states"], st["parents"], out=st["outs"]))
    x, f, i, z = st["x"], st["f"], st["i"], st["z"]
    kw = dict(f_bias=st["f_bias"], i_bias=st["i_bias"])
    if op == "gated_token":
        out, state = sgr.gated_scan_step(st["state0"], x[0], f[0], None if i is None else i[0],
                                         None if z is None else z[0],
                                         new_state=st["new_state"], **kw)
        return [out.unsqueeze(0), state]
    kw.update(lengths=st["lengths"])
    train = op == "gated_train"
    out, state, saved, _ = sgr.gated_scan_forward(x, f, i, z, state0=st["state0"], save=train, **kw)
    if not train:
        return [out, state]
    g = sgr.gated_scan_backward(x, f, saved, st["grad_out"], i, z, grad_state=st["grad_state"],
                                **kw)
    return [out, state] + [g[k] for k in ("g_x", "g_f", "g_f_bias", "g_state0", "g_i", "g_i_bias",
                                          "g_z") if k in g]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "clip":
        return _plain_clip(state)
    if op == "beam_select":
        return _plain_select(state)
    if op == "beam_reorder":
        return _plain_reorder(state)
    return _plain_gated(state, op == "gated_train")


# ------------------------------------------------------- the exact definition

def _exact_gated(st, train):
    """One step after the other, each row up to its own length; gradients by
    differentiating that program."""
    case = st["case"]
    T, B, D = case["T"], case["B"], case["D"]
    names = ["x", "f", "f_bias", "state0"] + (["i", "i_bias"] if case["input_gate"] else []) + \
        (["z"] if case["z"] else [])
    leaf = {k: st[k].double().contiguous().requires_grad_(train) for k in names}
    lens = _lengths(case)
    length = torch.tensor(lens, device="cuda").unsqueeze(-1)
    keep = torch.sigmoid(leaf["f"] + leaf["f_bias"])
    take = torch.sigmoid(leaf["i"] + leaf["i_bias"]) if case["input_gate"] else \
        torch.sigmoid(-leaf["f"] - leaf["f_bias"])
    new = take * leaf["x"]
    h, hs = leaf["state0"], []
    for t, (k, n) in enumerate(zip(keep.unbind(0), new.unbind(0))):
        if t >= max(lens):
            break
        nxt = k * h + n
        h = torch.where(t < length, nxt, h) if case["ragged"] else nxt
        hs.append(h)
    steps = len(hs)
    y = torch.stack(hs) if hs else leaf["x"][:0]
    if case["z"]:
        y = y * torch.nn.functional.silu(leaf["z"][:steps])
    if case["ragged"]:
        runs = torch.arange(steps, device="cuda")[:, None] < length.view(1, B)
        y = y * runs.unsqueeze(-1)
    out = torch.cat([y, torch.zeros(T - steps, B, D, dtype=torch.float64, device="cuda")])
    if not train:
        return [out, h]
    grads = torch.autograd.grad([out, h], [leaf[k] for k in names],
                                [st["grad_out"].double(), st["grad_state"].double()])
    return [out.detach(), h.detach()] + list(grads)


def _exact_clip(st):
    flat = torch.cat([t.double() for t in st["grads"]])
    norm = torch.linalg.vector_norm(flat)
    if norm.item() > st["max_norm"]:
        flat = flat * (st["max_norm"] / norm)
    return [norm.view(1)] + list(flat.split([t.numel() for t in st["grads"]]))


def _exact_select(st):
    """The scores in order, by sorting all candidates of each text."""
    case = st["case"]
    K, V, done = case["K"], case["V"], _done(case)
    best = []
    for b in range(case["B"]):
        rows = []
        for k in range(K):
            s = st["scores"][b, k].double()
            rows.append(s.view(1) if done[b][k] else
                        s + torch.log_softmax(st["logits"][b, k].double(), -1))
        best.append(torch.cat(rows).sort(descending=True).values[:K])
    return [torch.stack(best)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        return _exact_clip(st)
    if case["op"] == "beam_select":
        return _exact_select(st)
    if case["op"] == "beam_reorder":
        return [t.double().index_select(0, torch.cat([p + b * case["K"] for b, p in
                                                      enumerate(st["parents"])]))
                for t in st["states"]]
    return _exact_gated(st, case["op"] == "gated_train")
