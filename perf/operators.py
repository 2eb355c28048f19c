"""Cases and plain forms of the low-rank adapter operators and of gradient clipping.

`listed()` and `draw()` give cases, `prepare()` a user's inputs on the GPU,
`run()` one pass (the plain form in elementary torch operations, or the calls
of the package where `own` is true), `exact()` the same outputs in float64
from the definition, and `work()` the bytes and operations of a pass.

Activations are feature-major (features x tokens), as in the sparse layer of
the package.  A request is a run of consecutive tokens with one adapter (or
none); the adapters of a pool are stacked: A [n, rank, in], B [n, out, rank].
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ----------------------------------------------------------------- cases --

def _layer(name, op, dtype, tokens, requests, adapters, rank, n_in, n_out, ragged_ranks=False):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "requests": requests,
            "adapters": adapters, "rank": rank, "in": n_in, "out": n_out,
            "ragged_ranks": ragged_ranks}


def _clip(name, dtype, tensors, size, max_norm, spread):
    return {"name": name, "op": "clip", "dtype": dtype, "tensors": tensors, "size": size,
            "max_norm": max_norm, "spread": spread}


def listed():
    return [
        # one request decoding one token beside a 4096 x 4096 projection
        _layer("add-decode-1", "add", "bf16", 1, 1, 8, 16, 4096, 4096),
        # a decode batch: 64 requests of one token over a pool of 32 adapters
        _layer("add-decode-64", "add", "bf16", 64, 64, 32, 16, 4096, 11008),
        # a mixed batch of prompts of odd lengths, adapters of unequal ranks
        _layer("add-ragged-f16", "add", "f16", 2011, 37, 16, 32, 4096, 4096, True),
        # long prompts with wide adapters: the largest forward
        _layer("add-prompt", "add", "bf16", 8192, 8, 4, 64, 4096, 11008),
        # one adapter in training on 4096 tokens (packed sequences)
        _layer("backward-one", "backward", "bf16", 4096, 4, 1, 16, 4096, 4096),
        # several adapters trained in one batch, odd token count
        _layer("backward-ragged-f16", "backward", "f16", 2047, 23, 6, 32, 4096, 11008, True),
        # a full-precision run on a small layer
        _layer("backward-f32", "backward", "f32", 512, 3, 2, 8, 2048, 2048),
        # serving: one token of one request through W and its adapter
        _layer("project-1", "project", "bf16", 1, 1, 8, 16, 4096, 4096),
        # serving: a batch of 32 requests, one token each, wide output
        _layer("project-32-f16", "project", "f16", 32, 32, 16, 16, 4096, 11008),
        # the factors of a few dozen adapted layers
        _clip("clip-factors", "bf16", 48, 65536, 1.0, False),
        # value vectors, factors and norms of very unequal sizes, two formats
        _clip("clip-mixed", "mixed", 200, 450888, 1.0, True),
        # dense gradients of a few large layers, already below the limit
        _clip("clip-dense", "f32", 6, 11008 * 4096, 1.0e6, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add", "add", "backward", "project", "clip"])
    if op == "clip":
        dtype = rng.choice(["f32", "f16", "bf16", "mixed"])
        tensors = _log_int(rng, 1, 300)
        size = _log_int(rng, 1000, min(11008 * 4096, 200_000_000 // tensors))
        return {"op": op, "dtype": dtype, "tensors": tensors, "size": size,
                "max_norm": rng.choice([0.5, 1.0, 1.0e6]), "spread": rng.random() < 0.5}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    tokens = _log_int(rng, 1, 64 if op == "project" else 8192 if op == "add" else 4096)
    if dtype == "f32":
        tokens = min(tokens, 4096)
    requests = tokens if rng.random() < 0.3 and tokens <= 256 else _log_int(rng, 1, min(tokens, 64))
    return {"op": op, "dtype": dtype, "tokens": tokens, "requests": requests,
            "adapters": _log_int(rng, 1, 32), "rank": rng.choice([1, 4, 8, 16, 16, 24, 32, 64, 17]),
            "in": _log_int(rng, 256, 4096) if rng.random() < 0.5 else 64 * _log_int(rng, 4, 64),
            "out": _log_int(rng, 256, 11008) if rng.random() < 0.5 else 64 * _log_int(rng, 4, 172),
            "ragged_ranks": rng.random() < 0.3}


def _sizes(case):
    """Lengths of a clip case's tensors: equal, or spread down to a few
    hundred elements, odd ones among them."""
    n, size = case["tensors"], case["size"]
    if not case["spread"]:
        return [size] * n
    return [max(1, int(size * 2.0 ** (-(11.0 * i) / n)) - i % 3) for i in range(n)]


def _formats(case):
    if case["dtype"] == "mixed":
        return ["bf16" if i % 2 else "f32" for i in range(case["tensors"])]
    return [case["dtype"]] * case["tensors"]


# ---------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, std, dtype):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    if case["op"] == "clip":
        sizes, formats = _sizes(case), _formats(case)
        total = sum(sizes)
        # gradients whose norm is about 3, so that a limit of 0.5 or 1 clips
        grads = [normal((s,), 3.0 / math.sqrt(total), DTYPES[f]) for s, f in zip(sizes, formats)]
        # the clipped gradients go into one bucket per format
        buckets = {f: torch.empty(sum(s for s, h in zip(sizes, formats) if h == f),
                                  dtype=DTYPES[f], device="cuda") for f in sorted(set(formats))}
        at, out = dict.fromkeys(buckets, 0), []
        for s, f in zip(sizes, formats):
            out.append(buckets[f][at[f]:at[f] + s])
            at[f] += s
        return {"case": case, "grads": grads, "formats": formats, "out": out,
                "buckets": [buckets[f] for f in sorted(buckets)]}

    dt, T, S, n, R = (DTYPES[case["dtype"]], case["tokens"], case["requests"], case["adapters"],
                      case["rank"])
    n_in, n_out = case["in"], case["out"]
    # request lengths: every request at least one token, the rest at random
    cuts = torch.randperm(T - 1, generator=g, device="cuda")[:S - 1].sort().values + 1
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
    adapter = torch.randint(0, n, (S,), generator=g, device="cuda", dtype=torch.int32)
    # one request in eight of a batch runs on the base weights alone
    adapter[7::8] = -1
    ranks = (torch.randint(1, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
             if case["ragged_ranks"] else None)
    state = {"case": case, "offsets": offsets, "adapter": adapter, "ranks": ranks,
             "scale": torch.rand(n, generator=g, device="cuda") * 1.5 + 0.5,
             "A": normal((n, R, n_in), n_in ** -0.5, dt),
             "B": normal((n, n_out, R), R ** -0.5, dt),
             "xt": normal((n_in, T), 1.0, dt)}
    if case["op"] == "add":
        state["yt"] = normal((n_out, T), 1.0, dt)
    elif case["op"] == "backward":
        state["dyt"] = normal((n_out, T), 1.0 / math.sqrt(T), dt)
    else:
        state["W"] = normal((n_out, n_in), n_in ** -0.5, dt)
    return state


# ------------------------------------------------------------- one pass --

def _token_mask(s, T):
    """[n * R, T] truth values: adapter row j acts on token t."""
    n, R, _ = s["A"].shape
    token_request = torch.bucketize(torch.arange(T, device="cuda", dtype=torch.int32),
                                    s["offsets"][1:], right=True)
    of_token = s["adapter"][token_request]
    row = torch.arange(n * R, device="cuda")
    mask = (row // R)[:, None] == of_token[None, :]
    if s["ranks"] is not None:
        mask &= ((row % R) < s["ranks"][row // R])[:, None]
    return mask


def _plain_layer(s):
    case, dt = s["case"], s["A"].dtype
    n, R, n_in = s["A"].shape
    T = s["xt"].shape[1]
    mask = _token_mask(s, T)
    A = s["A"].float().reshape(n * R, n_in)
    B = s["B"].float().permute(1, 0, 2).reshape(-1, n * R)
    x = s["xt"].float()
    scale = s["scale"].repeat_interleave(R)[:, None]
    zero = x.new_zeros(())
    u = torch.where(mask, A @ x, zero) * scale
    if case["op"] == "backward":
        dy = s["dyt"].float()
        du = torch.where(mask, B.t() @ dy, zero) * scale
        dx = A.t() @ du
        dA = (du @ x.t()).reshape(n, R, n_in)
        dB = (dy @ u.t()).reshape(-1, n, R).permute(1, 0, 2)
        return dx.to(dt), dA.to(dt), dB.to(dt).contiguous()
    base = s["yt"].float() if case["op"] == "add" else s["W"].float() @ x
    return (base + B @ u).to(dt)


def _plain_clip(s):
    flat = torch.cat([g.float() for g in s["grads"]])
    norm = flat.square().sum(dtype=torch.float64).sqrt().float()
    coef = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    parts = torch.split(flat * coef, [g.numel() for g in s["grads"]])
    return [norm] + [torch.cat([p for p, f in zip(parts, s["formats"]) if f == name])
                     .to(DTYPES[name]) for name in sorted(set(s["formats"]))]


def run(state):
    op = state["case"]["op"]
    if own:
        import unstructured_sparse_linear_amd as S
        if op == "clip":
            norm = S.clip_grad_norm(state["grads"], state["case"]["max_norm"], out=state["out"])
            return [norm] + state["buckets"]
        args = (state["xt"], state["A"], state["B"], state["offsets"], state["adapter"],
                state["scale"], state["ranks"])
        if op == "add":
            return S.low_rank_add(state["yt"], *args)
        if op == "backward":
            return S.low_rank_backward(state["dyt"], *args)
        return S.low_rank_project(state["W"], *args)
    return _plain_clip(state) if op == "clip" else _plain_layer(state)


# ------------------------------------------------------- the definition --

def exact(case, seed):
    """Request by request in float64."""
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in s["grads"]))
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        return [torch.tensor(norm, dtype=torch.float64)] + [
            torch.cat([g.double() * coef for g, f in zip(s["grads"], s["formats"]) if f == name])
            for name in sorted(set(s["formats"]))]
    A, B, x = s["A"].double(), s["B"].double(), s["xt"].double()
    offsets, adapter, scale = s["offsets"].tolist(), s["adapter"].tolist(), s["scale"].tolist()
    ranks = s["ranks"].tolist() if s["ranks"] is not None else [case["rank"]] * case["adapters"]
    if case["op"] == "backward":
        dy = s["dyt"].double()
        dx, dA, dB = torch.zeros_like(x), torch.zeros_like(A), torch.zeros_like(B)
    elif case["op"] == "add":
        y = s["yt"].double()
    else:
        y = torch.mm(s["W"].double(), x)
    for i, a in enumerate(adapter):
        t = slice(offsets[i], offsets[i + 1])
        if a < 0:
            continue
        k = ranks[a]
        Aa, Ba, xs = A[a, :k], B[a, :, :k], x[:, t]
        u = torch.mm(Aa, xs)
        if case["op"] == "backward":
            du = scale[a] * torch.mm(Ba.t().contiguous(), dy[:, t])
            dx[:, t] = torch.mm(Aa.t().contiguous(), du)
            dA[a, :k] += torch.mm(du, xs.t().contiguous())
            dB[a, :, :k] += scale[a] * torch.mm(dy[:, t], u.t().contiguous())
        else:
            y[:, t] += scale[a] * torch.mm(Ba, u)
    return (dx, dA, dB) if case["op"] == "backward" else y


def work(case):
    if case["op"] == "clip":
        sizes, formats = _sizes(case), _formats(case)
        total = sum(s * BYTES[f] for s, f in zip(sizes, formats))
        return {"bytes": 2 * total, "flops": 3 * sum(sizes)}
    e, T, R, n_in, n_out = (BYTES[case["dtype"]], case["tokens"], case["rank"], case["in"],
                            case["out"])
    used = min(case["adapters"], case["requests"])
    factors = used * R * (n_in + n_out)
    if case["op"] == "add":
        return {"bytes": e * (T * (n_in + 2 * n_out) + factors),
                "flops": 2 * T * R * (n_in + n_out)}
    if case["op"] == "backward":
        grads = case["adapters"] * R * (n_in + n_out)
        return {"bytes": e * (T * (2 * n_in + n_out) + factors + grads),
                "flops": 2 * T * R * (3 * n_in + 2 * n_out)}
    return {"bytes": e * (n_in * n_out + T * (n_in + n_out) + factors),
            "flops": 2 * T * (n_in * n_out + R * (n_in + n_out))}
