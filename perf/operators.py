"""Workloads of the token-model operators: the gated linear recurrence (whole sequences, a training
pass, one decode step), the embedding lookup and its gradient, and sampling from logits.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU, ``run`` is one pass in the
plain form (elementary torch operations in 32 bits) or, where ``own`` is true, through the library,
``exact`` is the same from the definition in 64 bits, and ``work`` is what one pass has to move and
compute.

The recurrence, per batch row and channel (sigma: logistic function, kappa = c softplus(lam)):
    l_t = -kappa sigma(gate_a_t),   a_t = e^{l_t},   s_t = sqrt(1 - a_t^2)
    h_t = a_t h_{t-1} + s_t sigma(gate_x_t) u_t        (a reset token: a_t = 0, s_t = 1)
    out_t = h_t SiLU(z_t)                              (without z: out_t = h_t)
The lookup: out_i = scale * weight[ids_i], a negative id (padding) gives a row of zeros and no gradient.
Sampling, per row: logits / temperature, then the top_k largest, of those the shortest prefix (in falling
order) that holds top_p of their mass, of those the ones with at least min_p times the largest
probability; the token is the argmax of weight / noise with Exp(1) noise, which draws each kept token
with its probability; ties go to the lowest index; temperature 0 takes the largest logit.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DECAY_C = 8.0


def _seq(name, kind, batch, length, dim, io, z, h0, reset):
    return {"name": name, "kind": kind, "batch": batch, "length": length, "dim": dim, "io": io, "z": z, "h0": h0,
            "reset": reset}


def _emb(name, kind, count, vocab, dim, io, zipf):
    return {"name": name, "kind": kind, "count": count, "vocab": vocab, "dim": dim, "io": io, "zipf": zipf}


def _smp(name, rows, vocab, io, filters):
    return {"name": name, "kind": "sample", "rows": rows, "vocab": vocab, "io": io, "filters": filters}


def listed():
    return [
        # one sequence generating a token: the latency of a call
        _seq("step_1x2560", "step", 1, 1, 2560, "bf16", True, True, False),
        # 256 sequences generating a token each, the decode workload's batch and width
        _seq("step_256x5120", "step", 256, 1, 5120, "bf16", True, True, False),
        # reading four prompts at the widest layer
        _seq("scan_4x4096x5120", "scan", 4, 4096, 5120, "bf16", True, False, False),
        # one document of a million tokens with resets, few channels: the sequence has to be split
        _seq("scan_1x1048576x256", "scan", 1, 1048576, 256, "f32", False, True, True),
        # a training pass of a small layer over packed documents
        _seq("train_8x2048x1536", "train", 8, 2048, 1536, "bf16", True, False, True),
        # a training pass at odd sizes, continued from a state
        _seq("train_3x1537x1101", "train", 3, 1537, 1101, "f32", False, True, False),
        # the tokens of a training batch, word frequencies falling as in text
        _emb("lookup_16384x2560", "lookup", 16384, 50000, 2560, "bf16", True),
        # their gradient: few ids own most rows, most rows of the table get none
        _emb("grad_16384x2560", "lookup_grad", 16384, 50000, 2560, "bf16", True),
        # a short fine-tuning batch
        _emb("grad_777x768", "lookup_grad", 777, 32000, 768, "f32", False),
        # one sequence, every filter: the latency of a token
        _smp("sample_1x50000", 1, 50000, "bf16", "all"),
        # a large serving batch with the nucleus filter alone
        _smp("sample_256x128000", 256, 128000, "f32", "top_p"),
        # temperature alone, every token stays a candidate, odd row length
        _smp("sample_64x50001", 64, 50001, "bf16", "none"),
    ]


def _log_uniform(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["step", "scan", "scan", "train", "train", "lookup", "lookup_grad", "lookup_grad", "sample",
                       "sample"])
    io = rng.choice(["f32", "bf16"])
    if kind == "sample":
        c = _smp("", _log_uniform(rng, 1, 256), _log_uniform(rng, 1000, 128000), io,
                 rng.choice(["none", "top_k", "top_p", "all"]))
    elif kind in ("lookup", "lookup_grad"):
        dim = _log_uniform(rng, 64, 5120)
        c = _emb("", kind, _log_uniform(rng, 1, 32768), _log_uniform(rng, 1000, min(128000, 128000000 // dim)), dim,
                 io, rng.random() < 0.7)
    else:
        dim = _log_uniform(rng, 48, 5120)
        if rng.random() < 0.6:
            dim = (dim + 15) // 16 * 16
        batch = _log_uniform(rng, 1, 256 if kind == "step" else 8)
        length = 1 if kind == "step" else _log_uniform(rng, 2, max(2, min(65536, 25000000 // (batch * dim))))
        c = _seq("", kind, batch, length, dim, io, rng.random() < 0.5, kind == "step" or rng.random() < 0.5,
                 rng.random() < 0.4)
    c.pop("name")
    return c


# ------------------------------------------------------------------------------------------- inputs


def _zipf_weights(vocab):
    return 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    kind, dt = case["kind"], DTYPES[case["io"]]
    st = {"kind": kind, "dtype": dt}
    if kind in ("step", "scan", "train"):
        b, n, d = case["batch"], case["length"], case["dim"]
        shape = (b, d) if kind == "step" else (b, n, d)
        for name in ("u", "gate_a", "gate_x"):
            st[name] = normal(*shape).to(dt)
        # decays e^-kappa between 0.9 and 0.999 per channel at an open gate
        kappa = -torch.log(0.9 + 0.099 * uniform(d))
        st["lam"] = torch.log(torch.expm1(kappa / DECAY_C))
        st["z"] = normal(*shape).to(dt) if case["z"] else None
        st["h0"] = normal(b, d) if case["h0"] else None
        st["reset"] = (uniform(*shape[:-1]) < 1.0 / 256).to(torch.uint8) if case["reset"] else None
        if kind == "train":
            st["dout"] = normal(*shape).to(dt)
            st["dlast"] = normal(b, d) if case["h0"] else None
    elif kind in ("lookup", "lookup_grad"):
        n, v, d = case["count"], case["vocab"], case["dim"]
        if case["zipf"]:
            cdf = torch.from_numpy(np.cumsum(_zipf_weights(v))).to("cuda", torch.float64)
            rank = torch.searchsorted(cdf, uniform(n).double() * cdf[-1]).clamp(max=v - 1)
            ids = torch.randperm(v, generator=g, device="cuda")[rank]
        else:
            ids = torch.randint(v, (n,), generator=g, device="cuda")
        st["ids"] = torch.where(uniform(n) < 0.02, torch.full_like(ids, -1), ids)
        st["vocab"], st["scale"] = v, math.sqrt(d)
        if kind == "lookup":
            st["weight"] = (normal(v, d) / math.sqrt(d)).to(dt)
        else:
            st["dout"] = normal(n, d).to(dt)
    else:
        r, v, f = case["rows"], case["vocab"], case["filters"]
        st["logits"] = (normal(r, v) * (2.0 + 3.0 * uniform(r, 1))).to(dt)
        st["noise"] = torch.empty((r, v), device="cuda").exponential_(generator=g)
        temperature = 0.6 + 0.7 * uniform(r)
        st["temperature"] = torch.where(uniform(r) < 0.1, torch.zeros_like(temperature), temperature)
        st["top_k"] = torch.randint(20, 200, (r,), generator=g, device="cuda", dtype=torch.int32) \
            if f in ("top_k", "all") else None
        st["top_p"] = 0.8 + 0.19 * uniform(r) if f in ("top_p", "all") else None
        st["min_p"] = 0.02 * uniform(r) if f == "all" else None
        st["vocab"] = v
    return st


# ---------------------------------------------------------------------------------------- one pass


def run(st):
    if own:
        return _run_library(st)
    kind = st["kind"]
    if kind in ("step", "scan", "train"):
        return _plain_recurrence(st)
    if kind == "lookup":
        keep = (st["ids"] >= 0).unsqueeze(1)
        rows = st["weight"][st["ids"].clamp(min=0)].float() * st["scale"]
        return {"out": torch.where(keep, rows, torch.zeros_like(rows)).to(st["dtype"])}
    if kind == "lookup_grad":
        keep = st["ids"] >= 0
        grad = torch.zeros((st["vocab"], st["dout"].shape[1]), device="cuda")
        rows = torch.where(keep.unsqueeze(1), st["dout"].float(), torch.zeros((), device="cuda"))
        grad.index_add_(0, st["ids"].clamp(min=0), rows)
        return {"dweight": (grad * st["scale"]).to(st["dtype"])}
    return _plain_sample(st)


def _run_library(st):
    import selective_state_space_22_amd as lib

    kind = st["kind"]
    if kind == "step":
        out = lib.mamba_gated_state_update(st["h0"], st["u"], st["gate_a"], st["gate_x"], st["lam"], z=st["z"],
                                           reset=st["reset"], c=DECAY_C)
        return {"out": out, "state": st["h0"]}
    if kind == "scan":
        out, last = lib.mamba_gated_scan_fwd(st["u"], st["gate_a"], st["gate_x"], st["lam"], z=st["z"], h0=st["h0"],
                                             reset=st["reset"], c=DECAY_C)
        return {"out": out, "last_state": last}
    if kind == "train":
        out, last, states = lib.mamba_gated_scan_fwd(st["u"], st["gate_a"], st["gate_x"], st["lam"], z=st["z"],
                                                     h0=st["h0"], reset=st["reset"], c=DECAY_C, return_states=True)
        grads = lib.mamba_gated_scan_bwd(st["u"], st["gate_a"], st["gate_x"], st["lam"], st["dout"], z=st["z"],
                                         h0=st["h0"], reset=st["reset"], c=DECAY_C, states=states,
                                         dlast_state=st["dlast"])
        return {"out": out, "last_state": last, **{k: grads[k] for k in _GRADS if k in grads}}
    if kind == "lookup":
        return {"out": lib.mamba_embed_fwd(st["ids"], st["weight"], scale=st["scale"])}
    if kind == "lookup_grad":
        return {"dweight": lib.mamba_embed_bwd(st["ids"], st["dout"], st["vocab"], scale=st["scale"])}
    token, logprob = lib.mamba_sample(st["logits"], st["noise"], temperature=st["temperature"], top_k=st["top_k"],
                                      top_p=st["top_p"], min_p=st["min_p"])
    return {"token": token, "logprob": logprob}


_GRADS = ("du", "dgate_a", "dgate_x", "dlam", "dz", "dh0")


def _scan_by_doubling(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along dim 1, combining spans of doubled length each pass."""
    a, h, span = a.clone(), b.clone(), 1
    while span < a.shape[1]:
        h[:, span:] += a[:, span:] * h[:, :-span]
        a[:, span:] = a[:, span:] * a[:, :-span]
        span *= 2
    return h


def _plain_recurrence(st):
    step = st["kind"] == "step"
    u, ra, rx = (st[k].float().unsqueeze(1) if step else st[k].float() for k in ("u", "gate_a", "gate_x"))
    kappa = DECAY_C * torch.nn.functional.softplus(st["lam"])
    sig_a, sig_x = torch.sigmoid(ra), torch.sigmoid(rx)
    log_a = -kappa * sig_a
    a, s = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    live = None
    if st["reset"] is not None:
        live = (st["reset"].unsqueeze(1) if step else st["reset"]).unsqueeze(-1) == 0
        a, s = torch.where(live, a, torch.zeros_like(a)), torch.where(live, s, torch.ones_like(s))
    b = s * sig_x * u
    if st["h0"] is not None:
        b[:, 0] += a[:, 0] * st["h0"]
    h = _scan_by_doubling(a, b)
    gate = None
    if st["z"] is not None:
        z = st["z"].float().unsqueeze(1) if step else st["z"].float()
        gate = z * torch.sigmoid(z)
    out = (h if gate is None else h * gate).to(st["dtype"])
    if step:
        st["h0"].copy_(h[:, 0])
        return {"out": out[:, 0], "state": st["h0"]}
    last = h[:, -1].clone()
    if st["kind"] == "scan":
        return {"out": out, "last_state": last}
    dout = st["dout"].float()
    dh = dout if gate is None else dout * gate
    if st["dlast"] is not None:
        dh = dh.clone()
        dh[:, -1] += st["dlast"]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    grad = _scan_by_doubling(after.flip(1), dh.flip(1)).flip(1)
    start = torch.zeros_like(last) if st["h0"] is None else st["h0"]
    before = torch.cat([start.unsqueeze(1), h[:, :-1]], 1)
    # d(a h + s i u) / d(log a), times log a: the shared factor of the gradients at gate_a and lam
    e = grad * (a * before * log_a - a * a * sig_x * u * (log_a / s))
    if live is not None:
        e = torch.where(live, e, torch.zeros_like(e))
    dt = st["dtype"]
    grads = {"du": (grad * s * sig_x).to(dt), "dgate_a": (e * (1 - sig_a)).to(dt),
             "dgate_x": (grad * s * u * sig_x * (1 - sig_x)).to(dt),
             "dlam": e.sum((0, 1)) * DECAY_C * torch.sigmoid(st["lam"]) / kappa}
    if gate is not None:
        sig_z = torch.sigmoid(z)
        grads["dz"] = (dout * h * sig_z * (1 + z * (1 - sig_z))).to(dt)
    grads["dh0"] = a[:, 0] * grad[:, 0]
    return {"out": out, "last_state": last, **grads}


def _plain_sample(st):
    x = st["logits"].float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    top = x.max(1, keepdim=True).values
    t = st["temperature"].unsqueeze(1)
    scaled = torch.where(x == top, torch.zeros_like(x), (x - top) / torch.where(t > 0, t, torch.ones_like(t)))
    weight = torch.exp(scaled)
    weight, order = weight.sort(dim=1, descending=True, stable=True)
    rank = torch.arange(weight.shape[1], device="cuda")
    k = torch.full_like(t, weight.shape[1]).long() if st["top_k"] is None else st["top_k"].long().unsqueeze(1)
    k = torch.where(t > 0, torch.where(k > 0, k, torch.full_like(k, weight.shape[1])), torch.ones_like(k))
    weight = torch.where(rank < k, weight, torch.zeros_like(weight))
    if st["top_p"] is not None:
        p = st["top_p"].unsqueeze(1)
        upto = weight.cumsum(1)
        inside = (upto - weight < p * upto[:, -1:]) | (p >= 1)
        weight = torch.where(inside, weight, torch.zeros_like(weight))
    if st["min_p"] is not None:
        weight = torch.where(weight >= st["min_p"].unsqueeze(1), weight, torch.zeros_like(weight))
    kept = torch.zeros_like(weight).scatter_(1, order, weight)
    score = torch.where(kept > 0, kept / st["noise"], torch.full_like(kept, -1.0))
    best = score.max(1, keepdim=True).values
    token = torch.where(score == best, rank, weight.shape[1]).min(1).values
    logprob = scaled.gather(1, token.unsqueeze(1)).squeeze(1) - torch.log(kept.sum(1))
    return {"token": token, "logprob": logprob}


# ---------------------------------------------------------------------------- the definition in 64 bits


def _exact_scan(a, b):
    """h_t = a_t h_{t-1} + b_t from zero, token after token inside blocks of the sequence (all blocks at
    once), then block after block; differentiable."""
    batch, n, d = a.shape
    size = max(1, int(math.sqrt(n)))
    blocks = -(-n // size)
    pad = blocks * size - n
    if pad:
        a = torch.cat([a, a.new_ones((batch, pad, d))], 1)
        b = torch.cat([b, b.new_zeros((batch, pad, d))], 1)
    a, b = a.view(batch, blocks, size, d), b.view(batch, blocks, size, d)
    h, run_a, local, decay = b.new_zeros((batch, blocks, d)), b.new_ones((batch, blocks, d)), [], []
    for j in range(size):
        h, run_a = a[:, :, j] * h + b[:, :, j], run_a * a[:, :, j]
        local.append(h)
        decay.append(run_a)
    carry, entry = b.new_zeros((batch, d)), []
    for j in range(blocks):
        entry.append(carry)
        carry = run_a[:, j] * carry + h[:, j]
    entry = torch.stack(entry, 1)
    full = torch.stack([x + y * entry for x, y in zip(local, decay)], 2)
    return full.reshape(batch, blocks * size, d)[:, :n]


def _exact_recurrence(case, st):
    step = case["kind"] == "step"
    if case["batch"] * case["length"] * case["dim"] > (300e6 if case["kind"] == "scan" else 100e6):
        return None
    leaf = {k: (st[k].double().unsqueeze(1) if step else st[k].double()) for k in ("u", "gate_a", "gate_x", "z")
            if st[k] is not None}
    leaf["lam"] = st["lam"].double()
    leaf["h0"] = torch.zeros((case["batch"], case["dim"]), device="cuda", dtype=torch.float64) \
        if st["h0"] is None else st["h0"].double()
    train = case["kind"] == "train"
    if train:
        leaf = {k: v.requires_grad_() for k, v in leaf.items()}
    rate = DECAY_C * torch.log1p(torch.exp(leaf["lam"]))
    log_a = -rate / (1 + torch.exp(-leaf["gate_a"]))
    decay, root = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    if st["reset"] is not None:
        cut = (st["reset"].unsqueeze(1) if step else st["reset"]).unsqueeze(-1) != 0
        decay, root = decay.masked_fill(cut, 0.0), root.masked_fill(cut, 1.0)
    given = root * leaf["u"] / (1 + torch.exp(-leaf["gate_x"]))
    first = torch.cat([(given[:, 0] + decay[:, 0] * leaf["h0"]).unsqueeze(1), given[:, 1:]], 1)
    h = _exact_scan(decay, first)
    out = h if "z" not in leaf else h * leaf["z"] / (1 + torch.exp(-leaf["z"]))
    if step:
        return {"out": out[:, 0], "state": h[:, 0]}
    if not train:
        return {"out": out, "last_state": h[:, -1]}
    total = (out * st["dout"].double()).sum()
    if st["dlast"] is not None:
        total = total + (h[:, -1] * st["dlast"].double()).sum()
    names = [k for k in ("u", "gate_a", "gate_x", "lam", "z", "h0") if k in leaf]
    grads = torch.autograd.grad(total, [leaf[k] for k in names])
    return {"out": out.detach(), "last_state": h[:, -1].detach(), **{"d" + k: v for k, v in zip(names, grads)}}


def _exact_sample(case, st):
    logits, noise = st["logits"].double().cpu().numpy(), st["noise"].double().cpu().numpy()
    want = {k: None if st[k] is None else st[k].cpu().numpy().astype(np.float64)
            for k in ("temperature", "top_k", "top_p", "min_p")}
    token, logprob = np.zeros(case["rows"], np.int64), np.zeros(case["rows"])
    for r in range(case["rows"]):
        t = want["temperature"][r]
        y = logits[r] / t if t > 0 else np.where(np.arange(case["vocab"]) == np.argmax(logits[r]), 0.0, -np.inf)
        p = np.exp(y - y.max())
        by_size = np.lexsort((np.arange(case["vocab"]), -logits[r]))
        if want["top_k"] is not None and want["top_k"][r] > 0:
            by_size = by_size[: int(want["top_k"][r])]
        if want["top_p"] is not None and want["top_p"][r] < 1:
            held = np.cumsum(p[by_size])
            by_size = by_size[: 1 + int(np.searchsorted(held, want["top_p"][r] * held[-1], side="left"))]
        if want["min_p"] is not None:
            by_size = by_size[p[by_size] >= want["min_p"][r]]
        by_size = np.sort(by_size[p[by_size] > 0])
        token[r] = by_size[np.argmax(p[by_size] / noise[r, by_size])]
        logprob[r] = math.log(p[token[r]] / p[by_size].sum())
    return {"token": token, "logprob": logprob}


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("step", "scan", "train"):
        return _exact_recurrence(case, st)
    if kind == "sample":
        return _exact_sample(case, st)
    if kind == "lookup":
        padded = torch.cat([st["weight"].double() * st["scale"],
                            torch.zeros((1, case["dim"]), device="cuda", dtype=torch.float64)])
        return {"out": padded[torch.where(st["ids"] < 0, torch.full_like(st["ids"], case["vocab"]), st["ids"])]}
    # rows in id order, running sums over all of them, differences at the ends of each id's run
    order = torch.argsort(st["ids"])
    sums = torch.cat([torch.zeros((1, case["dim"]), device="cuda", dtype=torch.float64),
                      st["dout"].double()[order].cumsum(0)])
    ids = torch.arange(case["vocab"], device="cuda")
    ends = torch.searchsorted(st["ids"][order], torch.stack([ids, ids + 1]))
    return {"dweight": (sums[ends[1]] - sums[ends[0]]) * st["scale"]}


# ------------------------------------------------------------------------------------- what a pass needs


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    kind = case["kind"]
    if kind in ("step", "scan", "train"):
        state = case["batch"] * case["dim"]
        n = state * case["length"]
        tokens, z = case["batch"] * case["length"], int(case["z"])
        read = (3 + z) * n * e + case["dim"] * 4 + tokens * int(case["reset"]) + state * 4 * int(case["h0"])
        total = read + n * e + 4 * state
        flops = (20 + 5 * z) * n
        if kind == "train":
            total += read + n * e + state * 4 * int(case["h0"]) + (3 + z) * n * e + 4 * case["dim"] + 4 * state
            flops += (45 + 10 * z) * n
        return {"bytes": total, "flops": flops}
    if kind in ("lookup", "lookup_grad"):
        n, v, d = case["count"], case["vocab"], case["dim"]
        if kind == "lookup_grad":
            return {"bytes": n * 8 + n * d * e + v * d * e, "flops": n * d}
        w = _zipf_weights(v) if case["zipf"] else np.ones(v)
        distinct = float(np.sum(-np.expm1(0.98 * n * np.log1p(-w / w.sum()))))
        return {"bytes": n * 8 + n * d * e + distinct * d * e, "flops": n * d}
    r, v = case["rows"], case["vocab"]
    # noise is needed where a token stays: everywhere without filters, else for few
    noise = {"none": 4 * v, "top_p": 0, "top_k": 800, "all": 800}[case["filters"]]
    return {"bytes": r * (v * e + noise + 28), "flops": 6 * r * v}
