"""The operators of a fine-tuning or serving step over a frozen 8-bit base weight, as cases to measure.

  quantise       a weight to 8-bit floating point (e4m3) with one power-of-two scale per 128 x 128 block, in both orientations
  forward        the multi-adapter LoRA layer over that weight, the rows of X quantised with one scale per 128 columns
  train          that forward, then dA, dB and the input gradient over the same 8-bit weight
  orthogonalise  Newton-Schulz orthogonalisation of every listed adapter's rank rows
  step           momentum, orthogonalisation and the in-place update of both factors of every listed adapter

Where `own` is false `run` computes each in elementary torch operations; where it is true it calls the library.
"""
import math

import torch

own = False

QMAX = 448.0                              # largest e4m3 value
COEF = (3.4445, -4.7750, 2.0315)          # quintic Newton-Schulz coefficients
STEPS = 5
EPS = 1e-7
MU, LR, DECAY = 0.95, 0.02, 0.01
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a small fp32 layer, its widths odd multiples of 64 (the last scale block is half empty)
        {"name": "quantise_704x576_f32", "op": "quantise", "d_in": 576, "d_out": 704, "dtype": "f32"},
        # the up projection of the fine-tuning workload, requantised after a merge
        {"name": "quantise_11008x4096", "op": "quantise", "d_in": 4096, "d_out": 11008, "dtype": "bf16"},
        # one request decoding: a single token
        {"name": "forward_1_token", "op": "forward", "T": 1, "K": 1, "d_in": 4096, "d_out": 4096, "N": 64,
         "lo": 16, "hi": 16, "dtype": "bf16", "runs": False},
        # a decode batch, every token its own adapter
        {"name": "forward_64_tokens", "op": "forward", "T": 64, "K": 1, "d_in": 4096, "d_out": 4096, "N": 64,
         "lo": 16, "hi": 16, "dtype": "bf16", "runs": False},
        # a serving batch over adapters of irregular ranks
        {"name": "forward_256_mixed_ranks", "op": "forward", "T": 256, "K": 1, "d_in": 4096, "d_out": 11008,
         "N": 256, "lo": 8, "hi": 128, "dtype": "bf16", "runs": False},
        # prefill of a few long requests: contiguous runs of tokens per adapter
        {"name": "forward_8192_prefill", "op": "forward", "T": 8192, "K": 1, "d_in": 4096, "d_out": 11008, "N": 4,
         "lo": 16, "hi": 16, "dtype": "bf16", "runs": True},
        # a small fp32 training step with two gated adapters per token
        {"name": "train_333_top2_f32", "op": "train", "T": 333, "K": 2, "d_in": 576, "d_out": 1344, "N": 24,
         "lo": 2, "hi": 16, "dtype": "f32", "runs": False},
        # the fine-tuning workload: forward and backward of one projection, dropout on the adapters' input
        {"name": "train_8192", "op": "train", "T": 8192, "K": 1, "d_in": 4096, "d_out": 11008, "N": 4,
         "lo": 16, "hi": 16, "dtype": "bf16", "runs": True},
        # the gradients of four rank-16 adapters: latency
        {"name": "orthogonalise_4_rank16", "op": "orthogonalise", "M": 4, "N": 4, "lo": 16, "hi": 16, "d": 4096},
        # a fleet trained together, ranks up to 128
        {"name": "orthogonalise_64_mixed", "op": "orthogonalise", "M": 64, "N": 80, "lo": 8, "hi": 128, "d": 11008},
        # the optimiser step after train_8192
        {"name": "step_4_rank16", "op": "step", "M": 4, "N": 4, "lo": 16, "hi": 16, "d_in": 4096, "d_out": 11008,
         "dtype": "bf16"},
        # many adapters of small irregular ranks
        {"name": "step_256_mixed", "op": "step", "M": 256, "N": 300, "lo": 2, "hi": 64, "d_in": 5120, "d_out": 5120,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return 64 * max(1, _log(rng, lo // 64, hi // 64))


def draw(rng):
    op = rng.choice(["quantise", "forward", "forward", "train", "orthogonalise", "step"])
    if op == "quantise":
        return {"op": op, "d_in": _width(rng, 576, 4096), "d_out": _width(rng, 576, 11008),
                "dtype": rng.choice(["bf16", "f32"])}
    if op in ("forward", "train"):
        T = _log(rng, 1 if op == "forward" else 64, 8192)
        dtype = "f32" if T < 1024 and rng.random() < 0.25 else "bf16"
        c = {"op": op, "T": T, "K": rng.choice([1, 1, 2]), "d_in": _width(rng, 576, 4096),
             "d_out": _width(rng, 576, 11008 if dtype == "bf16" else 2048), "N": rng.randint(2, 96), "lo": 2,
             "hi": 0, "dtype": dtype, "runs": T >= 1024}
        c["hi"] = rng.choice([16, 32, 64] if T < 1024 else [8, 16])
        if c["runs"]:
            c["K"], c["N"] = 1, rng.randint(2, 8)
        return c
    M = _log(rng, 2, 48)
    hi = rng.choice([8, 16, 33, 64, 128])
    c = {"op": op, "M": M, "N": M + rng.randint(0, 8), "lo": rng.randint(1, hi), "hi": hi}
    if op == "orthogonalise":
        return dict(c, d=_width(rng, 1024, 11008))
    return dict(c, d_in=_width(rng, 1024, 5120), d_out=_width(rng, 1024, 5120), dtype=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _pool(g, case, seed):
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
            "scale": (0.5 + torch.rand(N, generator=g, device=DEV)), "max_rank": hi}


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


def _up(d):
    return (d + 127) // 128 * 128


def _exponents(amax):
    """The smallest e >= -126 with amax <= 448 * 2^e, for finite amax."""
    m, ex = torch.frexp(amax)
    e = ex.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)


def _power(e):
    """2^e in fp32 for -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise_weight(W):
    """Codes [d_out][up(d_in)] and exponents [blocks of d_out][blocks of d_in] of W [d_out][d_in]."""
    o, i = W.shape
    P = torch.zeros(_up(o), _up(i), device=W.device)
    P[:o, :i] = W.float()
    B = P.view(_up(o) // 128, 128, _up(i) // 128, 128)
    e = _exponents(B.abs().amax(dim=(1, 3)))
    C = (B * _power(-e)[:, None, :, None]).view_as(P).to(torch.float8_e4m3fn)
    return C[:o].contiguous(), e


def _scale_rows(e):
    """Exponents as the bytes e + 127, rows padded to a multiple of four."""
    n = (e.shape[1] + 3) // 4 * 4
    out = torch.zeros(e.shape[0], n, dtype=torch.uint8, device=e.device)
    out[:, : e.shape[1]] = (e + 127).to(torch.uint8)
    return out


def _turned(C, d_in, d_out):
    """The codes of W^T, [d_in][up(d_out)], from those of W."""
    Q = torch.zeros(d_in, _up(d_out), dtype=torch.uint8, device=C.device)
    Q[:, :d_out] = C.view(torch.uint8)[:, :d_in].t()
    return Q.view(torch.float8_e4m3fn)


def _gradient_pages(g, n, d):
    """Rows whose sizes fall off over three decades and that lean on each other, as the rows of a gradient do."""
    rows = _normal(g, n, d) * (10.0 ** (-3.0 * torch.rand(n, 1, generator=g, device=DEV)))
    return rows + 0.3 * rows.roll(1, 0)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "quantise":
        o, i = case["d_out"], case["d_in"]
        # trained weights: rows of unlike size
        W = _normal(g, o, i, std=math.sqrt(0.02)) * torch.exp(_normal(g, o, 1, std=0.5))
        return {"case": case, "W_t": W.to(DTYPES[case["dtype"]])}
    s = dict(_pool(g, case, seed), case=case)
    P = s["n_pages"]
    if op in ("forward", "train"):
        dt, d_in, d_out = DTYPES[case["dtype"]], case["d_in"], case["d_out"]
        s["X"] = _normal(g, case["T"], d_in, dtype=dt)
        s["X"][:, 5::97] *= 16                                    # a few columns much larger than the rest
        s["codes"], e = _quantise_weight(_normal(g, d_out, d_in, std=math.sqrt(0.02)))
        s["scales"] = _scale_rows(e)
        s["a_pages"] = _normal(g, P, d_in, std=1 / 8, dtype=dt)
        s["b_pages"] = _normal(g, P, d_out, std=math.sqrt(0.02), dtype=dt)
        s["ids"], s["gates"] = _routing(g, case)
        s["mask"], s["keep"] = None, 1.0
        if op == "train":
            s["turned"] = _turned(s["codes"], d_in, d_out)
            s["scales_t"] = _scale_rows(e.t())
            s["mask"] = (torch.rand(case["T"], d_in, generator=g, device=DEV) < 0.9).to(torch.uint8)
            s["keep"] = float(torch.tensor(1 / 0.9, dtype=torch.float32))
            s["dY"] = _normal(g, case["T"], d_out, dtype=dt)
            s["dA"] = torch.zeros(P, d_in, device=DEV)
            s["dB"] = torch.zeros(P, d_out, device=DEV)
        return s
    cpu = torch.Generator().manual_seed(seed * 31 + 5)
    s["adapters"] = torch.randperm(case["N"], generator=cpu)[: case["M"]].to(torch.int32).to(DEV)
    if op == "orthogonalise":
        s["src"] = _gradient_pages(g, P, case["d"])
        s["out"] = torch.zeros(P, case["d"], device=DEV)
        return s
    for f, d in (("a", case["d_in"]), ("b", case["d_out"])):
        s["grad_" + f] = _gradient_pages(g, P, d)
        s["mom_" + f] = 5 * _gradient_pages(g, P, d)
        s["master_" + f] = _normal(g, P, d, std=1 / 8)
        s["pages_" + f] = s["master_" + f].to(DTYPES[case["dtype"]])
    return s


# ---------------------------------------------------------------- plain forms

def _quantised_rows(x):
    """x with every 128 columns of a row rounded to e4m3 under their own power-of-two scale (fp32 values)."""
    T, d = x.shape
    B = torch.zeros(T, _up(d), device=x.device)
    B[:, :d] = x.float()
    B = B.view(T, -1, 128)
    e = _exponents(B.abs().amax(dim=2, keepdim=True))
    return ((B * _power(-e)).to(torch.float8_e4m3fn).float() * _power(e)).view(T, -1)


def _weight_values(codes, scales):
    n = codes.shape[1] // 128
    s = _power(scales[:, :n].to(torch.int32) - 127).repeat_interleave(128, 0)[: codes.shape[0]]
    return (codes.float().view(codes.shape[0], n, 128) * s[:, :, None]).view(codes.shape[0], -1)


def _owners(s):
    """The adapter that owns each page (N: none)."""
    N = s["rank"].numel()
    own_ = torch.full((s["n_pages"],), N, dtype=torch.int64, device=DEV)
    own_[s["page_ids"].long()] = torch.repeat_interleave(torch.arange(N, device=DEV), s["rank"].long())
    return own_


def _weights_of_pages(s):
    """[T][pages]: gate x scale of the token's slot that has the page's adapter, else 0."""
    N, T = s["rank"].numel(), s["ids"].shape[0]
    C = torch.zeros(T, N + 1, device=DEV)
    live = s["ids"] >= 0
    at = torch.where(live, s["ids"], torch.full_like(s["ids"], N)).long()
    C.scatter_add_(1, at, torch.where(live, s["gates"] * s["scale"][at.clamp(max=N - 1)], torch.zeros_like(s["gates"])))
    C[:, N] = 0
    return C[:, _owners(s)]


def _plain_forward(s):
    d_in = s["case"]["d_in"]
    X = s["X"].float()
    Xm = X if s["mask"] is None else X * s["mask"].float()
    C = _weights_of_pages(s) * s["keep"]
    U = (Xm @ s["a_pages"].float().t()) * C
    Y = _quantised_rows(s["X"]) @ _weight_values(s["codes"], s["scales"]).t() + U @ s["b_pages"].float()
    return Y.to(s["X"].dtype), U, C, Xm


def _plain_train(s):
    Y, U, C, Xm = _plain_forward(s)
    dY = s["dY"].float()
    G = (dY @ s["b_pages"].float().t()) * C
    s["dA"].copy_(G.t() @ Xm)
    s["dB"].copy_(U.t() @ dY)
    dX = _quantised_rows(s["dY"]) @ _weight_values(s["turned"], s["scales_t"]).t()
    dX = dX + s["mask"].float() * (G @ s["a_pages"].float())
    return Y, s["dA"], s["dB"], dX.to(s["X"].dtype)


def _rows_of(s):
    """Page of every rank row of the listed adapters [M][max_rank], and which of them exist."""
    a = s["adapters"].long()
    j = torch.arange(s["max_rank"], device=DEV)
    live = j[None] < s["rank"].long()[a][:, None]
    at = (s["page_start"].long()[a][:, None] + j[None]).clamp(max=s["page_ids"].numel() - 1)
    return s["page_ids"].long()[at], live


def _newton_schulz(X):
    a, b, c = COEF
    X = X / (X.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


def _plain_orthogonalise(s):
    pid, live = _rows_of(s)
    X = _newton_schulz(s["src"][pid] * live[:, :, None])
    s["out"][pid[live]] = X[live]
    return s["out"]


def _plain_step_of(s, f):
    pid, live = _rows_of(s)
    G = s["grad_" + f][pid] * live[:, :, None]
    mom = MU * s["mom_" + f][pid] * live[:, :, None] + G
    O = _newton_schulz(G + MU * mom)
    rows = pid[live]
    s["mom_" + f][rows] = mom[live]
    s["master_" + f][rows] = s["master_" + f][rows] * (1 - LR * DECAY) - LR * O[live]
    s["pages_" + f][rows] = s["master_" + f][rows].to(s["pages_" + f].dtype)


# ---------------------------------------------------------------- one pass

def _stepped(s):
    return [s[k + f] for f in ("a", "b") for k in ("mom_", "master_", "pages_")]


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "quantise":
        C, e = _quantise_weight(s["W_t"])
        d_out, d_in = s["W_t"].shape
        return C, _turned(C, d_in, d_out), _scale_rows(e), _scale_rows(e.t())
    if op == "forward":
        return _plain_forward(s)[0]
    if op == "train":
        return _plain_train(s)
    if op == "orthogonalise":
        return _plain_orthogonalise(s)
    _plain_step_of(s, "a")
    _plain_step_of(s, "b")
    return _stepped(s)


def _kept(s, name, make):
    """A buffer that a program keeps from call to call."""
    if name not in s:
        s[name] = make()
    return s[name]


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def _own_pool(s, B, a_pages, b_pages):
    return B.Pool(B.LORA_BF16 if a_pages.dtype == torch.bfloat16 else B.LORA_F32, a_pages.shape[1], b_pages.shape[1],
                  a_pages, b_pages, s["rank"], s["page_start"], s["page_ids"], s["scale"])


def _own(s, op):
    from lora_adapter_amd import binding as B
    c = s["case"]
    if op == "quantise":
        d_out, d_in = s["W_t"].shape
        w = _kept(s, "w", lambda: B.QuantisedWeight.empty(d_out, d_in, DEV))
        B.lora_quantise_weight(s["W_t"], B.LORA_BF16 if c["dtype"] == "bf16" else B.LORA_F32, w)
        return w.q_t.view(torch.float8_e4m3fn), w.q.view(torch.float8_e4m3fn), w.scale, w.scale_t
    if op in ("forward", "train"):
        T, K, d_in, d_out, N, R = c["T"], c["K"], c["d_in"], c["d_out"], c["N"], s["max_rank"]
        pool = _kept(s, "pool", lambda: _own_pool(s, B, s["a_pages"], s["b_pages"]))
        w = _kept(s, "w", lambda: B.QuantisedWeight(d_out, d_in, s["codes"], s["scales"], s.get("turned"),
                                                    s.get("scales_t")))
        plan = _kept(s, "plan", lambda: _bytes(B.lora_plan_bytes(T, K, N)))
        ws = _kept(s, "ws", lambda: _bytes(B.lora_apply_quantised_workspace_bytes(T, K, d_in, d_out, R, pool.dtype)))
        Y = torch.empty(T, d_out, dtype=s["X"].dtype, device=DEV)
        B.lora_forward_quantised(s["ids"], s["gates"], T, K, s["X"], w, Y, s["mask"], s["keep"], pool, plan, ws)
        if op == "forward":
            return Y
        gws = _kept(s, "gws", lambda: _bytes(B.lora_grad_workspace_bytes(T, K, N, d_in, d_out, R, pool.dtype)))
        xws = _kept(s, "xws", lambda: _bytes(B.lora_grad_x_quantised_workspace_bytes(T, d_in, d_out, pool.dtype)))
        dX = torch.empty(T, d_in, dtype=s["X"].dtype, device=DEV)
        B.lora_grad(s["X"], s["mask"], s["keep"], s["dY"], T, K, s["gates"], pool, plan, ws, s["dA"], s["dB"], R, gws)
        B.lora_grad_x_quantised(s["dY"], w, s["mask"], T, K, pool, plan, gws, R, dX, xws)
        return Y, s["dA"], s["dB"], dX
    M, R = c["M"], s["max_rank"]
    if op == "orthogonalise":
        pool = _kept(s, "pool", lambda: _own_pool(s, B, s["src"], s["src"]))
        ws = _kept(s, "ws", lambda: _bytes(B.lora_orthogonalise_workspace_bytes(M, R, c["d"])))
        B.lora_orthogonalise(pool, s["adapters"], M, R, s["src"], s["out"], c["d"], STEPS, COEF, EPS, ws)
        return s["out"]
    pool = _kept(s, "pool", lambda: _own_pool(s, B, s["pages_a"], s["pages_b"]))
    ws = _kept(s, "ws", lambda: _bytes(B.lora_orthogonal_step_workspace_bytes(M, R, c["d_in"], c["d_out"])))
    fa, fb = _kept(s, "factors", lambda: tuple(
        B.FactorUpdate(s["pages_" + f], s["grad_" + f], s["mom_" + f], s["master_" + f], LR, DECAY) for f in "ab"))
    B.lora_orthogonal_step(pool, s["adapters"], M, R, fa, fb, MU, True, STEPS, COEF, EPS, ws)
    return _stepped(s)


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "quantise":
        n = case["d_in"] * case["d_out"]
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + 2), "flops": 2 * n}
    r = (case["lo"] + case["hi"]) / 2
    if op in ("forward", "train"):
        T, K, i, o = case["T"], case["K"], case["d_in"], case["d_out"]
        e = 2 if case["dtype"] == "bf16" else 4
        used = case["N"] * (1 - (1 - 1 / case["N"]) ** (T * K))
        factors = used * r * (i + o)
        lora = 2 * T * K * r * (i + o)
        b, f = T * (i + o) * e + i * o + factors * e, 2 * T * i * o + lora
        if op == "train":       # dY read, dX written, W^T read, the mask read, dA and dB written
            b += T * (i + o) * e + i * o + T * i + factors * 4
            f += 2 * T * i * o + 3 * lora
        return {"bytes": b, "flops": f}
    rows = case["M"] * r
    if op == "orthogonalise":
        return {"bytes": rows * case["d"] * 8, "flops": 4 * rows * r * case["d"]}
    d = case["d_in"] + case["d_out"]
    return {"bytes": rows * d * (4 + 8 + 8 + (2 if case["dtype"] == "bf16" else 4)), "flops": 4 * rows * r * d}


# ---------------------------------------------------------------- 64 bits

def _exact_blocks(V):
    """V [n][m] (each row one scale block), rounded to e4m3 under the block's scale: values over the scale, and e."""
    top = V.abs().amax(dim=1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / QMAX))
    e = torch.where(top > QMAX * torch.exp2(e), e + 1, e)
    e = torch.where(top <= QMAX * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 0, e, torch.full_like(e, -126.0)).clamp(min=-126.0)
    v = V / torch.exp2(e)[:, None]
    mag = torch.floor(torch.log2(torch.where(v == 0, torch.ones_like(v), v.abs()))).clamp(min=-6.0)
    q = torch.exp2(mag - 3)
    return torch.round(v / q) * q, e


def _exact_rows(x):
    """The quantised rows' values."""
    T, d = x.shape
    full, rest = d // 128, d % 128
    parts = []
    if full:
        v, e = _exact_blocks(x[:, : 128 * full].double().reshape(-1, 128))
        parts.append((v * torch.exp2(e)[:, None]).reshape(T, -1))
    if rest:
        v, e = _exact_blocks(x[:, 128 * full:].double())
        parts.append(v * torch.exp2(e)[:, None])
    return torch.cat(parts, 1)


def _exact_weight(codes, scales, rows, cols):
    W = codes[:, :cols].double()
    for b in range((cols + 127) // 128):
        e = scales[:, b].double() - 127
        W[:, 128 * b: 128 * b + 128] *= torch.exp2(e)[torch.arange(rows, device=DEV) // 128][:, None]
    return W


def _exact_layer(s):
    c = s["case"]
    train = c["op"] == "train"
    Y = _exact_rows(s["X"]) @ _exact_weight(s["codes"], s["scales"], c["d_out"], c["d_in"]).t()
    X = s["X"].double() if s["mask"] is None else s["X"].double() * s["mask"].double()
    dA = dB = dX = dY = None
    if train:
        dY = s["dY"].double()
        dX = _exact_rows(s["dY"]) @ _exact_weight(s["turned"], s["scales_t"], c["d_in"], c["d_out"]).t()
        dA, dB = s["dA"].double(), s["dB"].double()
    for a in torch.unique(s["ids"]).tolist():
        if a < 0:
            continue
        t, k = torch.nonzero(s["ids"] == a, as_tuple=True)
        p = s["page_ids"][int(s["page_start"][a]): int(s["page_start"][a + 1])].long()
        A, Bm = s["a_pages"][p].double(), s["b_pages"][p].double()
        w = (s["gates"][t, k].double() * s["scale"][a].double() * s["keep"])[:, None]
        U = (X[t] @ A.t()) * w
        Y[t] += U @ Bm
        if train:
            G = (dY[t] @ Bm.t().contiguous()) * w
            dA[p], dB[p] = G.t() @ X[t], U.t() @ dY[t]
            dX[t] += s["mask"][t].double() * (G @ A)
    return (Y, dA, dB, dX) if train else Y


def _exact_factor(N):
    """The orthogonalised N: its left singular vectors, with the polynomial's value in place of each singular value."""
    n = torch.sqrt((N * N).sum()) + EPS
    w, V = torch.linalg.eigh((N @ N.t() / (n * n)).cpu())
    f = torch.ones_like(w)
    for _ in range(STEPS):
        p = COEF[0] + COEF[1] * w + COEF[2] * w * w
        f, w = f * p, w * p * p
    return ((V * f) @ V.t()).to(N.device) @ N / n


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        W = s["W_t"].double()
        o, i = W.shape
        V = torch.zeros(_up(o), _up(i), dtype=torch.float64, device=DEV)
        V[:o, :i] = W
        no, ni = V.shape[0] // 128, V.shape[1] // 128
        v, e = _exact_blocks(V.view(no, 128, ni, 128).permute(0, 2, 1, 3).reshape(no * ni, -1))
        v = v.view(no, ni, 128, 128).permute(0, 2, 1, 3).reshape(V.shape)
        vt = v.t()[:i].contiguous()
        vt[:, o:] = 0
        return v[:o].contiguous(), vt, None, None
    if op in ("forward", "train"):
        return _exact_layer(s)
    rows = [s["page_ids"][int(s["page_start"][a]): int(s["page_start"][a + 1])].long() for a in s["adapters"].tolist()]
    if op == "orthogonalise":
        out = s["out"].double()
        for p in rows:
            out[p] = _exact_factor(s["src"][p].double())
        return out
    got = []
    for f in "ab":
        G, mom, P = s["grad_" + f].double(), s["mom_" + f].double(), s["master_" + f].double()
        pages = s["pages_" + f].double()
        for p in rows:
            mom[p] = MU * mom[p] + G[p]
            P[p] = P[p] * (1 - LR * DECAY) - LR * _exact_factor(G[p] + MU * mom[p])
            pages[p] = P[p]
        got += [mom, P, pages]
    return got
