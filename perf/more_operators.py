"""What a fine-tuning or serving step needs between and behind its adapter layers, as cases to measure.

  gated       the gated feed-forward block: both projections with their adapters, the activation and the product
  gated_grad  its backward: the gradients of both projections' results and of the block's input
  loss        softmax cross entropy of a large vocabulary (mode "grad": with the gradient of the hidden states)
  clip        every listed adapter's gradient norm over all layers, and the gradients clipped by it

Where `own` is false `run` computes each in elementary torch operations; where it is true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one request decoding: a single token
        {"name": "gated_1_token", "op": "gated", "T": 1, "K": 1, "d_in": 4096, "d_out": 11008, "N": 64, "lo": 16,
         "hi": 16, "dtype": "bf16", "runs": False, "act": "silu", "train": False},
        # a decode batch, two gated adapters of irregular ranks for each token
        {"name": "gated_48_top2", "op": "gated", "T": 48, "K": 2, "d_in": 4096, "d_out": 11008, "N": 64, "lo": 8,
         "hi": 64, "dtype": "bf16", "runs": False, "act": "gelu_tanh", "train": False},
        # a small fp32 block in training, its widths odd multiples of 64
        {"name": "gated_333_top2_f32", "op": "gated", "T": 333, "K": 2, "d_in": 576, "d_out": 1344, "N": 24, "lo": 2,
         "hi": 16, "dtype": "f32", "runs": False, "act": "gelu", "train": True},
        # a serving batch over many adapters of irregular ranks
        {"name": "gated_700_mixed_ranks", "op": "gated", "T": 700, "K": 1, "d_in": 2240, "d_out": 5824, "N": 96,
         "lo": 8, "hi": 64, "dtype": "bf16", "runs": False, "act": "silu", "train": False},
        # the fine-tuning workload's forward: what the backward needs is stored, dropout on the adapters' input
        {"name": "gated_8192_train", "op": "gated", "T": 8192, "K": 1, "d_in": 4096, "d_out": 11008, "N": 4, "lo": 16,
         "hi": 16, "dtype": "bf16", "runs": True, "act": "silu", "train": True},
        # the backward of a small batch with two adapters for each token
        {"name": "gated_grad_600_top2", "op": "gated_grad", "T": 600, "K": 2, "d_in": 2240, "d_out": 5824, "N": 32,
         "lo": 4, "hi": 32, "dtype": "bf16", "runs": False, "act": "gelu_tanh"},
        # the fine-tuning workload's backward
        {"name": "gated_grad_8192", "op": "gated_grad", "T": 8192, "K": 1, "d_in": 4096, "d_out": 11008, "N": 4,
         "lo": 16, "hi": 16, "dtype": "bf16", "runs": True, "act": "silu"},
        # scoring a text: the loss alone, no token ignored
        {"name": "loss_1024_eval", "op": "loss", "T": 1024, "V": 32000, "d": 4096, "dtype": "bf16", "ignored": 0.0,
         "mode": "eval"},
        # a small fp32 head with an odd vocabulary
        {"name": "loss_333_odd_f32", "op": "loss", "T": 333, "V": 5003, "d": 576, "dtype": "f32", "ignored": 0.25,
         "mode": "grad"},
        # the fine-tuning workload's loss: prompts are ignored, the rest gives a gradient
        {"name": "loss_8192_train", "op": "loss", "T": 8192, "V": 128256, "d": 4096, "dtype": "bf16", "ignored": 0.3,
         "mode": "grad"},
        # four rank-16 adapters on the seven projections of one layer: latency
        {"name": "clip_4_rank16", "op": "clip", "M": 4, "N": 4, "lo": 16, "hi": 16, "d": 4096, "F": 11008,
         "layers": 1, "together": False},
        # a fleet trained together, irregular ranks
        {"name": "clip_48_mixed", "op": "clip", "M": 48, "N": 56, "lo": 4, "hi": 64, "d": 4096, "F": 11008,
         "layers": 2, "together": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return 64 * max(1, _log(rng, lo // 64, hi // 64))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "loss", "loss", "clip"])
    if op in ("gated", "gated_grad"):
        T = _log(rng, 1 if op == "gated" else 16, 8192)
        dtype = "f32" if T < 1024 and rng.random() < 0.25 else "bf16"
        c = {"op": op, "T": T, "K": rng.choice([1, 1, 2]), "d_in": _width(rng, 576, 4096 if dtype == "bf16" else 1024),
             "d_out": _width(rng, 576, 11008 if dtype == "bf16" else 2048), "N": rng.randint(2, 96), "lo": 2,
             "hi": rng.choice([16, 32, 64] if T < 1024 else [8, 16]), "dtype": dtype, "runs": T >= 1024,
             "act": rng.choice(ACTS)}
        if c["runs"]:
            c["K"], c["N"] = 1, rng.randint(2, 8)
        return dict(c, train=rng.random() < 0.5) if op == "gated" else c
    if op == "loss":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        big = dtype == "bf16"
        return {"op": op, "T": _log(rng, 1, 8192 if big else 1024), "V": _log(rng, 1000, 128256 if big else 16000),
                "d": _width(rng, 256, 4096 if big else 1024), "dtype": dtype,
                "ignored": rng.choice([0.0, 0.3, 0.6]), "mode": rng.choice(["eval", "grad", "grad"])}
    M = _log(rng, 2, 32)
    hi = rng.choice([8, 16, 33, 64])
    return {"op": op, "M": M, "N": M + rng.randint(0, 8), "lo": rng.randint(1, hi), "hi": hi,
            "d": _width(rng, 1024, 4096), "F": _width(rng, 1024, 11008), "layers": rng.choice([1, 1, 2]),
            "together": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _tables(g, case, seed):
    """Ranks and a page table whose pages are scattered, three of them owned by no adapter."""
    N, lo, hi = case["N"], case["lo"], case["hi"]
    # the ranks go by the case alone, so that every seed has the same number of pages
    rank = torch.randint(lo, hi + 1, (N,), generator=torch.Generator().manual_seed(1000 * N + hi), dtype=torch.int32)
    cpu = torch.Generator().manual_seed(seed * 7919 + 13)
    start = torch.zeros(N + 1, dtype=torch.int32)
    start[1:] = torch.cumsum(rank, 0)
    total = int(start[-1])
    ids = torch.randperm(total + 3, generator=cpu)[:total].to(torch.int32)
    return {"rank": rank.to(DEV), "page_start": start.to(DEV), "page_ids": ids.to(DEV), "n_pages": total + 3,
            "max_rank": hi}


def _routing(g, case):
    T, K, N = case["T"], case["K"], case["N"]
    if case["runs"]:
        ids = (torch.arange(T, device=DEV) * N // T).to(torch.int32).reshape(T, 1)
    else:
        ids = torch.rand(T, N, generator=g, device=DEV).topk(K, dim=1).indices.to(torch.int32)
        gone = torch.rand(T, K, generator=g, device=DEV) < 0.03      # slots without an adapter
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    gates = torch.ones(T, K, device=DEV) if K == 1 else torch.softmax(_normal(g, T, K), dim=1)
    return ids.contiguous(), gates.contiguous()


def _prepare_gated(g, case, seed):
    s = dict(_tables(g, case, seed), case=case)
    T, d, F, P, dt = case["T"], case["d_in"], case["d_out"], s["n_pages"], DTYPES[case["dtype"]]
    for p in ("gate", "up"):
        s["a_" + p] = _normal(g, P, d, std=1 / 8, dtype=dt)
        s["b_" + p] = _normal(g, P, F, std=math.sqrt(0.02), dtype=dt)
        s["scale_" + p] = 0.5 + torch.rand(case["N"], generator=g, device=DEV)
    s["ids"], s["gates"] = _routing(g, case)
    s["mask"], s["keep"] = None, 1.0
    if case["op"] == "gated_grad" or case["train"]:
        s["mask"] = (torch.rand(T, d, generator=g, device=DEV) < 0.9).to(torch.uint8)
        s["keep"] = float(torch.tensor(1 / 0.9, dtype=torch.float32))
    std = math.sqrt(1 / d)
    if case["op"] == "gated":
        s["X"] = _normal(g, T, d, dtype=dt)
        s["X"][:, 5::97] *= 16                                    # a few columns much larger than the rest
        for p in ("gate", "up"):
            s["w_" + p] = _normal(g, F, d, std=std, dtype=dt)
        return s
    for p in ("gate", "up"):
        s["pre_" + p] = _normal(g, T, F, std=2.0, dtype=dt)       # what the forward stored
        s["w_" + p] = _normal(g, d, F, std=std, dtype=dt)         # the weights the other way round
    s["dH"] = _normal(g, T, F, std=0.01, dtype=dt)
    return s


def _prepare_loss(g, case):
    T, V, d, dt = case["T"], case["V"], case["d"], DTYPES[case["dtype"]]
    s = {"case": case, "W_t": _normal(g, V, d, std=math.sqrt(2 / d), dtype=dt)}
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    # hidden states that lean towards their target's row, some of them hard: losses from nearly nothing to the whole log
    lean = 14 * torch.rand(T, 1, generator=g, device=DEV)
    s["X"] = (_normal(g, T, d) + lean * s["W_t"][y].float() / math.sqrt(2)).to(dt)
    # requests of 64 tokens, the first part of each a prompt without a target
    prompt = (torch.arange(T, device=DEV) % 64) < int(round(64 * case["ignored"]))
    s["targets"] = torch.where(prompt & (T > 1), torch.full_like(y, -1), y).to(torch.int32)
    live = s["targets"] >= 0
    s["weights"] = (0.5 + torch.rand(T, generator=g, device=DEV)) / live.sum().clamp(min=1)
    return s


# the projections of a layer: how many of them, and their widths
def _projections(case):
    d, F, n = case["d"], case["F"], case["layers"]
    return {"attention": (4 * n, d, d), "up": (2 * n, d, F), "down": (n, F, d)}


def _prepare_clip(g, case, seed):
    s = dict(_tables(g, case, seed), case=case)
    P, N = s["n_pages"], case["N"]
    cpu = torch.Generator().manual_seed(seed * 31 + 5)
    s["adapters"] = torch.randperm(N, generator=cpu)[: case["M"]].to(torch.int32).to(DEV)
    # gradients of adapters of unlike size, so that some are clipped and some are not
    size = torch.exp(_normal(g, N + 1, 1))[_owners(s)]
    s["grads"], s["out"] = {}, {}
    for name, (n, d_in, d_out) in _projections(case).items():
        for f, w in (("A", d_in), ("B", d_out)):
            s["grads"][name + f] = torch.randn(n, P, w, generator=g, device=DEV).mul_(size / w)
            s["out"][name + f] = torch.zeros(n, P, w, device=DEV)
    # about the middle of the adapters' norms, and well under the norm of all of them
    mid = math.sqrt((case["lo"] + case["hi"]) / 2 * sum(n * (1 / i + 1 / o) for n, i, o in _projections(case).values()))
    s["max_norm"] = float(torch.tensor(mid, dtype=torch.float32))
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "loss":
        return _prepare_loss(g, case)
    if case["op"] == "clip":
        return _prepare_clip(g, case, seed)
    return _prepare_gated(g, case, seed)


# ---------------------------------------------------------------- plain forms

def _owners(s):
    """The adapter that owns each page (N: none)."""
    N = s["rank"].numel()
    own_ = torch.full((s["n_pages"],), N, dtype=torch.int64, device=DEV)
    own_[s["page_ids"].long()] = torch.repeat_interleave(torch.arange(N, device=DEV), s["rank"].long())
    return own_


def _weights_of_pages(s, scale):
    """[T][pages]: gate x scale x keep scale of the token's slot that has the page's adapter, else 0."""
    N, T = s["rank"].numel(), s["ids"].shape[0]
    C = torch.zeros(T, N + 1, device=DEV)
    live = s["ids"] >= 0
    at = torch.where(live, s["ids"], torch.full_like(s["ids"], N)).long()
    C.scatter_add_(1, at, torch.where(live, s["gates"] * scale[at.clamp(max=N - 1)], torch.zeros_like(s["gates"])))
    C[:, N] = 0
    return C[:, _owners(s)] * s["keep"]


def _act(name, x):
    """act(x) and act'(x)."""
    if name == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    if name == "gelu":
        p = 0.5 * torch.erfc(-x * math.sqrt(0.5))
        return x * p, p + x * torch.exp(-0.5 * x * x) * math.sqrt(0.5 / math.pi)
    c = math.sqrt(2 / math.pi)
    z = 2 * c * (x + 0.044715 * x ** 3)
    p = 1 / (1 + torch.exp(-z))                                   # (1 + tanh(z / 2)) / 2
    return x * p, p + x * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * x * x)


def _plain_projection(s, X, Xm, p):
    U = (Xm @ s["a_" + p].float().t()) * _weights_of_pages(s, s["scale_" + p])
    return X @ s["w_" + p].float().t() + U @ s["b_" + p].float()


def _plain_gated(s):
    dt = s["X"].dtype
    X = s["X"].float()
    Xm = X if s["mask"] is None else X * s["mask"].float()
    g, u = _plain_projection(s, X, Xm, "gate"), _plain_projection(s, X, Xm, "up")
    H = (_act(s["case"]["act"], g)[0] * u).to(dt)
    return (H, g.to(dt), u.to(dt)) if s["case"]["train"] else H


def _plain_back(s, dY, p):
    G = (dY @ s["b_" + p].float().t()) * _weights_of_pages(s, s["scale_" + p])
    return dY @ s["w_" + p].float().t() + s["mask"].float() * (G @ s["a_" + p].float())


def _plain_gated_grad(s):
    dt = s["dH"].dtype
    a, da = _act(s["case"]["act"], s["pre_gate"].float())
    dH = s["dH"].float()
    dg, du = dH * s["pre_up"].float() * da, dH * a
    return dg.to(dt), du.to(dt), (_plain_back(s, dg, "gate") + _plain_back(s, du, "up")).to(dt)


def _plain_loss(s):
    X, W, live = s["X"].float(), s["W_t"].float(), s["targets"] >= 0
    y = s["targets"].long().clamp(min=0)[:, None]
    w = torch.where(live, s["weights"], torch.zeros_like(s["weights"]))
    l = X @ W.t()
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - top)
    z = e.sum(dim=1, keepdim=True)
    loss = w * (torch.log(z) + top - l.gather(1, y))[:, 0]
    if s["case"]["mode"] == "eval":
        return loss
    e /= z
    e.scatter_add_(1, y, torch.full_like(z, -1.0))
    return loss, ((e @ W) * w[:, None]).to(s["X"].dtype)


def _slots(s):
    """The place of each page's adapter in the list (M: not listed)."""
    M, N = s["adapters"].numel(), s["rank"].numel()
    at = torch.full((N + 1,), M, dtype=torch.int64, device=DEV)
    at[s["adapters"].long()] = torch.arange(M, device=DEV)
    return at[_owners(s)]


def _plain_clip(s):
    M, slot = s["adapters"].numel(), _slots(s)
    of_page = sum(t.double().square().sum(dim=(0, 2)) for t in s["grads"].values())
    square = torch.zeros(M + 1, dtype=torch.float64, device=DEV).index_add_(0, slot, of_page)[:M]
    norm = torch.cat([square, square.sum()[None]]).sqrt()
    by = norm[M].expand(M) if s["case"]["together"] else norm[:M]
    coef = torch.cat([torch.where(by > s["max_norm"], s["max_norm"] / by, torch.ones_like(by)).float(),
                      torch.zeros(1, device=DEV)])[slot][:, None]
    live = (slot < M)[:, None]
    out = {k: torch.where(live, t * coef, s["out"][k]) for k, t in s["grads"].items()}
    return norm.float(), out


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "loss": _plain_loss, "clip": _plain_clip}[op](s)


# ---------------------------------------------------------------- the library's calls

def _kept(s, name, make):
    """A buffer that a program keeps from call to call."""
    if name not in s:
        s[name] = make()
    return s[name]


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def _pool(s, B, p):
    a, b = s["a_" + p], s["b_" + p]
    return B.Pool(B.LORA_BF16 if a.dtype == torch.bfloat16 else B.LORA_F32, a.shape[1], b.shape[1], a, b, s["rank"],
                  s["page_start"], s["page_ids"], s["scale_" + p])


def _own(s, op):
    from lora_adapter_amd import binding as B
    c = s["case"]
    if op in ("gated", "gated_grad"):
        T, K, d, F, N, R = c["T"], c["K"], c["d_in"], c["d_out"], c["N"], s["max_rank"]
        act = {"silu": B.LORA_ACT_SILU, "gelu": B.LORA_ACT_GELU, "gelu_tanh": B.LORA_ACT_GELU_TANH}[c["act"]]
        gate, up = _kept(s, "pools", lambda: (_pool(s, B, "gate"), _pool(s, B, "up")))
        plan = _kept(s, "plan", lambda: _bytes(B.lora_plan_bytes(T, K, N)))
        new = lambda n: torch.empty(T, n, dtype=gate.tensors[0].dtype, device=DEV)
        if op == "gated":
            wg, wu = _kept(s, "ws", lambda: [_bytes(B.lora_apply_workspace_bytes(T, K, d, F, R, gate.dtype))
                                             for _ in range(2)])
            H, g, u = new(F), new(F) if c["train"] else None, new(F) if c["train"] else None
            B.lora_gated_forward(s["ids"], s["gates"], T, K, s["X"], s["w_gate"], s["w_up"], act, H, g, u, s["mask"],
                                 s["keep"], gate, up, plan, wg, wu)
            return (H, g, u) if c["train"] else H
        if "planned" not in s:                                    # the forward's plan
            B.lora_plan(s["ids"], s["gates"], T, K, gate, plan)
            s["planned"] = True
        ws = _kept(s, "ws", lambda: _bytes(B.lora_gated_grad_workspace_bytes(T, K, d, F, R, gate.dtype)))
        dg, du, dX = new(F), new(F), new(d)
        B.lora_gated_grad(s["dH"], s["pre_gate"], s["pre_up"], act, s["w_gate"], s["w_up"], s["mask"], s["keep"], T, K,
                          s["gates"], gate, up, plan, R, dg, du, dX, ws)
        return dg, du, dX
    if op == "loss":
        T, V, d, grad = c["T"], c["V"], c["d"], c["mode"] == "grad"
        dt = B.LORA_BF16 if c["dtype"] == "bf16" else B.LORA_F32
        ws = _kept(s, "ws", lambda: _bytes(B.lora_cross_entropy_workspace_bytes(T, V, d, dt, grad)))
        loss = torch.empty(T, device=DEV)
        dX = torch.empty_like(s["X"]) if grad else None
        B.lora_cross_entropy(s["X"], s["W_t"], dt, T, V, d, s["targets"], s["weights"], 1.0, loss, dX, ws)
        return (loss, dX) if grad else loss
    M, R = c["M"], s["max_rank"]
    layers = _kept(s, "layers", lambda: _layers(s, B))
    ws = _kept(s, "ws", lambda: _bytes(B.lora_clip_grad_workspace_bytes(layers, M, R)))
    norm = torch.empty(M + 1, device=DEV)
    B.lora_clip_grad(layers, s["adapters"], M, R, s["max_norm"], c["together"], norm, ws)
    return norm, s["out"]


def _layers(s, B):
    one = torch.ones_like(s["rank"], dtype=torch.float32)
    got = []
    for name, (n, d_in, d_out) in _projections(s["case"]).items():
        a, b, oa, ob = (s[k][name + f] for k in ("grads", "out") for f in "AB")
        for i in range(n):
            pool = B.Pool(B.LORA_F32, d_in, d_out, a[i], b[i], s["rank"], s["page_start"], s["page_ids"], one)
            got.append((pool, a[i], b[i], oa[i], ob[i]))
    return B.GradLayers(got)


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "loss":
        T, V, d, e = case["T"] * (1 - case["ignored"]), case["V"], case["d"], 2 if case["dtype"] == "bf16" else 4
        grad = case["mode"] == "grad"
        return {"bytes": V * d * e + T * d * e * (2 if grad else 1) + 4 * case["T"],
                "flops": 2 * T * V * d * (2 if grad else 1)}
    r = (case["lo"] + case["hi"]) / 2
    if op == "clip":
        n = case["M"] * r * sum(n * (i + o) for n, i, o in _projections(case).values())
        return {"bytes": 8 * n, "flops": 3 * n}
    T, K, d, F = case["T"], case["K"], case["d_in"], case["d_out"]
    e = 2 if case["dtype"] == "bf16" else 4
    used = case["N"] * (1 - (1 - 1 / case["N"]) ** (T * K))
    factors, lora = 2 * used * r * (d + F), 4 * T * K * r * (d + F)
    if op == "gated":
        rows = T * (d + F * (3 if case["train"] else 1)) * e + (T * d if case["train"] else 0)
    else:               # dH and both stored results read, both gradients and dX written, the mask read
        rows = T * (d + 5 * F) * e + T * d
    return {"bytes": rows + 2 * d * F * e + factors * e, "flops": 4 * T * d * F + lora}


# ---------------------------------------------------------------- 64 bits

def _exact_act(name, x):
    if name == "silu":
        p = torch.sigmoid(x)
        return x * p, p + x * p * torch.sigmoid(-x)
    if name == "gelu":
        p = torch.special.ndtr(x)
        return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 3 * 0.044715 * x * x)


def _exact_adapters(s, p):
    """For every adapter in use: its tokens, their gates and scales, A and B."""
    for a in torch.unique(s["ids"]).tolist():
        if a < 0:
            continue
        t, k = torch.nonzero(s["ids"] == a, as_tuple=True)
        rows = s["page_ids"][int(s["page_start"][a]): int(s["page_start"][a + 1])].long()
        w = (s["gates"][t, k].double() * s["scale_" + p][a].double() * s["keep"])[:, None]
        yield t, w, s["a_" + p][rows].double(), s["b_" + p][rows].double()


def _exact_gated(s):
    X = s["X"].double()
    Xm = X if s["mask"] is None else X * s["mask"].double()
    got = []
    for p in ("gate", "up"):
        Y = X @ s["w_" + p].double().t()
        for t, w, A, Bm in _exact_adapters(s, p):
            Y[t] += ((Xm[t] @ A.t()) * w) @ Bm
        got.append(Y)
    H = _exact_act(s["case"]["act"], got[0])[0] * got[1]
    return (H, got[0], got[1]) if s["case"]["train"] else H


def _exact_gated_grad(s):
    a, da = _exact_act(s["case"]["act"], s["pre_gate"].double())
    dH = s["dH"].double()
    d = {"gate": dH * s["pre_up"].double() * da, "up": dH * a}
    dX = 0
    for p in ("gate", "up"):
        dX = dX + d[p] @ s["w_" + p].double().t()
        for t, w, A, Bm in _exact_adapters(s, p):
            dX[t] += s["mask"][t].double() * (((d[p][t] @ Bm.t()) * w) @ A)
    return d["gate"], d["up"], dX


def _exact_loss(s):
    """In pieces of the tokens: log-softmax, and its gradient by the formula."""
    T, grad = s["X"].shape[0], s["case"]["mode"] == "grad"
    W = s["W_t"].double()
    loss, dX = torch.zeros(T, dtype=torch.float64, device=DEV), torch.zeros(s["X"].shape, dtype=torch.float64, device=DEV)
    for t0 in range(0, T, 1024):
        y = s["targets"][t0: t0 + 1024].long()
        rows = torch.nonzero(y >= 0)[:, 0]
        L = torch.log_softmax(s["X"][t0 + rows].double() @ W.t(), dim=1)
        w = s["weights"][t0 + rows].double()
        loss[t0 + rows] = -w * L[torch.arange(rows.numel(), device=DEV), y[rows]]
        if grad:
            dX[t0 + rows] = w[:, None] * (torch.exp(L) @ W - W[y[rows]])
    return (loss, dX) if grad else loss


def _exact_clip(s):
    total, norms, pages = 0.0, [], []
    for a in s["adapters"].tolist():
        p = s["page_ids"][int(s["page_start"][a]): int(s["page_start"][a + 1])].long()
        sq = sum(float(torch.linalg.vector_norm(t[:, p].double())) ** 2 for t in s["grads"].values())
        norms.append(math.sqrt(sq))
        total += sq
        pages.append(p)
    out = {k: t.double() for k, t in s["out"].items()}
    for n, p in zip(norms, pages):
        n = math.sqrt(total) if s["case"]["together"] else n
        c = min(1.0, s["max_norm"] / n)
        for k, t in s["grads"].items():
            out[k][:, p] = t[:, p].double() * c
    return torch.tensor(norms + [math.sqrt(total)], dtype=torch.float64, device=DEV), out


def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "gated_grad": _exact_gated_grad, "loss": _exact_loss,
            "clip": _exact_clip}[case["op"]](s)
