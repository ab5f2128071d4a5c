"""The prompt-side operators of the quantised path: their measured cases, plain forms and 64-bit references.

A prompt goes through per-token INT8 quantisation and the INT8 W8A8 matmul, the per-head norms and rotary
positions of queries and keys, the store of keys and values into the quantised cache, and causal attention over
the packed prompt; the decode step afterwards makes the same calls with one token per sequence.
"""
import math

import torch

own = False

DEVICE = "cuda"
D_CACHE = 128  # head_dim of the quantised cache


# --------------------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------------------

# Forty-eight requests of a chat front end that arrive together: one token to a few hundred.
MIXED = ",".join(str(1 + (37 * i * i + 11 * i) % 331) for i in range(48))


def listed():
    return [
        # One token's activations before a projection of a decode step: launch latency.
        {"name": "tokens_decode", "op": "quantize_tokens", "rows": 1, "width": 8192, "type": "bf16", "pad": 0},
        # A packed prompt's activations before the down projection, rows of a wider buffer.
        {"name": "tokens_prompt", "op": "quantize_tokens", "rows": 8192, "width": 28672, "type": "bf16", "pad": 64},
        # The qkv projection of one token: the weights are read once.
        {"name": "matmul_token", "op": "matmul", "rows": 1, "outputs": 10240, "width": 8192},
        # The down projection of a decode batch that is not a multiple of any tile.
        {"name": "matmul_batch", "op": "matmul", "rows": 100, "outputs": 8192, "width": 28672},
        # The gate and up projection of a packed prompt: bound by the tensor cores.
        {"name": "matmul_prompt", "op": "matmul", "rows": 8190, "outputs": 57344, "width": 8192},
        # Norms and positions of a decode step: 128 sequences, contexts of up to 8,000 tokens.
        {"name": "rope_decode", "op": "norm_rope", "tokens": 128, "heads": 64, "kv_heads": 8, "dim": 128,
         "rotated": 128, "interleaved": False, "norm": True, "far": 8000},
        # The same over a packed prompt.
        {"name": "rope_prompt", "op": "norm_rope", "tokens": 16384, "heads": 64, "kv_heads": 8, "dim": 128,
         "rotated": 128, "interleaved": False, "norm": True, "far": 16384},
        # One new token for each of 128 sequences into the int4 cache; one in eight rows is padding.
        {"name": "store_decode", "op": "store", "form": "int4", "tokens": 128, "kv_heads": 8, "sequences": 128,
         "capacity": 1000, "padded": 8},
        # A packed prompt's keys and values into the fp8 cache.
        {"name": "store_prompt", "op": "store", "form": "fp8", "tokens": 16000, "kv_heads": 8, "sequences": 8,
         "capacity": 4000, "padded": 0},
        # Many short prompts in one pass.
        {"name": "attention_mixed", "op": "attention", "lengths": MIXED, "heads": 64, "kv_heads": 8, "dim": 128},
        # One long document.
        {"name": "attention_long", "op": "attention", "lengths": "16384", "heads": 64, "kv_heads": 8, "dim": 128},
        # A few prompts of ordinary length on a smaller geometry, five query heads to a key head.
        {"name": "attention_small_heads", "op": "attention", "lengths": "2048,1900,777,4001", "heads": 20,
         "kv_heads": 4, "dim": 64},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize_tokens", "matmul", "matmul", "norm_rope", "store", "attention", "attention"])
    if op == "quantize_tokens":
        width = 32 * _log(rng, 1, 896)
        rows = min(_log(rng, 1, 16384), 8192 * 28672 // width)
        return {"op": op, "rows": rows, "width": width, "type": rng.choice(["bf16", "f32"]),
                "pad": rng.choice([0, 8, 64])}
    if op == "matmul":
        width, outputs = 32 * _log(rng, 2, 896), _log(rng, 16, 57344)
        rows = min(_log(rng, 1, 8190), 8190 * 57344 * 8192 // (width * outputs))
        return {"op": op, "rows": rows, "outputs": outputs, "width": width}
    if op == "norm_rope":
        kv_heads, dim = rng.randint(1, 16), rng.choice([64, 128])
        heads = kv_heads * rng.randint(1, 8)
        tokens = min(_log(rng, 1, 16384), 16384 * 72 * 128 // ((heads + kv_heads) * dim))
        return {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rotated": rng.choice([dim, dim, dim // 2, 16]), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.7, "far": _log(rng, 1, 1000000)}
    if op == "store":
        sequences, kv_heads = _log(rng, 1, 128), rng.randint(1, 16)
        tokens = min(max(sequences, _log(rng, 1, 16000)), 16000 * 8 // kv_heads)
        return {"op": op, "form": rng.choice(["int4", "fp8"]), "tokens": tokens, "kv_heads": kv_heads,
                "sequences": sequences, "capacity": -(-tokens // sequences) + rng.randint(0, 500),
                "padded": rng.choice([0, 3, 8])}
    kv_heads, dim = rng.randint(1, 8), rng.choice([64, 128])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    longest, lengths = _log(rng, 1, 8192), []
    for _ in range(_log(rng, 1, 40)):
        lengths.append(rng.randint(0, longest))
    lengths[-1] = longest
    while sum(n * n for n in lengths) * kv_heads * group * dim > 16384 * 16384 * 64 * 128 // 2 or sum(lengths) > 40000:
        lengths = lengths[1:] if len(lengths) > 1 else [lengths[0] // 2]
    return {"op": op, "lengths": ",".join(map(str, lengths)), "heads": kv_heads * group, "kv_heads": kv_heads,
            "dim": dim}


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def work(case):
    op = case["op"]
    if op == "quantize_tokens":
        size = 4 if case["type"] == "f32" else 2
        values = case["rows"] * case["width"]
        return {"bytes": values * (size + 1) + 4 * case["rows"], "flops": 3 * values}
    if op == "matmul":
        m, n, k = case["rows"], case["outputs"], case["width"]
        return {"bytes": m * k + n * k + 2 * m * n + 4 * m + 2 * n, "flops": 2 * m * n * k}
    if op == "norm_rope":
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * values + 4 * case["tokens"] + 2 * case["rotated"] + 4 * case["dim"],
                "flops": 7 * values}
    if op == "store":
        vectors = 2 * case["tokens"] * case["kv_heads"]
        if case["padded"]:
            vectors -= 2 * ((case["tokens"] + case["padded"] - 1) // case["padded"]) * case["kv_heads"]
        stored = D_CACHE // 2 + 4 if case["form"] == "int4" else D_CACHE
        return {"bytes": max(vectors, 1) * (2 * D_CACHE + stored) + 8 * case["tokens"],
                "flops": 5 * max(vectors, 1) * D_CACHE}
    lengths = _lengths(case)
    total, pairs = sum(lengths), sum(n * (n + 1) // 2 for n in lengths)
    return {"bytes": 2 * total * case["dim"] * (2 * case["heads"] + 2 * case["kv_heads"]) + 4 * (len(lengths) + 1),
            "flops": 4 * case["dim"] * case["heads"] * pairs}


# --------------------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------------------

def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=dtype)


def _projection(g, tokens, heads, kv_heads, dim):
    """Queries, keys and values as a fused qkv projection leaves them: slices of one [tokens][...] buffer.  Keys
    have channels of larger magnitude and a mean away from zero, as trained models' do."""
    fused = _normal(g, tokens, heads + 2 * kv_heads, dim, dtype=torch.bfloat16)
    q, k, v = fused.split([heads, kv_heads, kv_heads], dim=1)
    k.mul_(1 + 2 * torch.rand(kv_heads, dim, generator=g, device=DEVICE).pow(4).to(torch.bfloat16))
    k.add_(_normal(g, kv_heads, dim, dtype=torch.bfloat16) * 0.5)
    return q, k, v


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    op = case["op"]
    state = {"case": case}
    if op == "quantize_tokens":
        rows, width = case["rows"], case["width"]
        dtype = torch.float32 if case["type"] == "f32" else torch.bfloat16
        x = _normal(g, rows, width + case["pad"], dtype=dtype)
        # one channel in a hundred carries activations twenty times as large
        x.mul_(1 + 19 * (torch.rand(width + case["pad"], generator=g, device=DEVICE) < 0.01).to(dtype))
        state["x"] = x[:, :width]
    elif op == "matmul":
        m, n, k = case["rows"], case["outputs"], case["width"]
        codes = lambda *s: torch.randint(-127, 128, s, generator=g, device=DEVICE, dtype=torch.int8)  # noqa: E731
        state["xq"], state["weight"] = codes(m, k), codes(n, k)
        state["xscales"] = torch.rand(m, generator=g, device=DEVICE) * 0.05 + 0.01
        state["scales"] = (torch.rand(n, generator=g, device=DEVICE) * 0.001 + 0.0002).to(torch.bfloat16)
    elif op == "norm_rope":
        state["q"], state["k"], _ = _projection(g, case["tokens"], case["heads"], case["kv_heads"], case["dim"])
        state["positions"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=DEVICE,
                                           dtype=torch.int32)
        pairs = torch.arange(case["rotated"] // 2, device=DEVICE, dtype=torch.float64)
        state["inv_freq"] = (500000.0 ** (-2 * pairs / case["rotated"])).float()
        weights = 1 + 0.2 * _normal(g, 2, case["dim"])
        state["weights"] = tuple(weights.to(torch.bfloat16).unbind(0)) if case["norm"] else (None, None)
    elif op == "store":
        tokens, heads = case["tokens"], case["kv_heads"]
        _, state["k"], state["v"] = _projection(g, tokens, heads, heads, D_CACHE)
        size = (case["sequences"], case["capacity"], heads)
        slots = torch.randperm(case["sequences"] * case["capacity"], generator=g, device=DEVICE)[:tokens]
        slots = slots.sort().values  # a prompt's tokens follow one another in their sequence's part of the cache
        if case["padded"]:
            slots[::case["padded"]] = -1
        state["slots"] = slots
        width = D_CACHE // 2 if case["form"] == "int4" else D_CACHE
        state["cache"] = {n: torch.zeros(*size, width, device=DEVICE, dtype=torch.uint8)
                          for n in ("k_codes", "v_codes")}
        if case["form"] == "int4":
            for n in ("k_scales", "k_zeros", "v_scales", "v_zeros"):
                state["cache"][n] = torch.zeros(*size, device=DEVICE, dtype=torch.bfloat16)
        else:
            state["k_scale"], state["v_scale"] = (torch.full((1,), s, device=DEVICE) for s in (0.031, 0.011))
    else:
        lengths = _lengths(case)
        state["q"], state["k"], state["v"] = _projection(g, sum(lengths), case["heads"], case["kv_heads"],
                                                         case["dim"])
        starts = [0]
        for n in lengths:
            starts.append(starts[-1] + n)
        state["spans"] = list(zip(starts[:-1], starts[1:]))
        state["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEVICE)
    return state


# --------------------------------------------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------------------------------------------

def _over(a, number):
    """a / number as a division: by a number on the host it may become a product with the reciprocal."""
    return a / a.new_full((), number)


def _plain_quantize_tokens(s):
    x = s["x"].float()
    scales = _over(x.abs().amax(dim=1), 127.0)
    scales = torch.where(scales == 0, torch.ones_like(scales), scales)
    return {"codes": torch.round(x / scales[:, None]).clamp(-127, 127).to(torch.int8), "scales": scales}


def _plain_matmul(s):
    y = s["xq"].float() @ s["weight"].float().t()
    return y.mul_(s["xscales"][:, None]).mul_(s["scales"].float()).to(torch.bfloat16)


def _plain_norm_rope(s):
    case = s["case"]
    angles = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angles.cos().float()[:, None], angles.sin().float()[:, None]

    def one(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * weight.float()
        turned, rest = x[..., :case["rotated"]], x[..., case["rotated"]:]
        if case["interleaved"]:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = turned.chunk(2, dim=-1)
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([turned, rest], dim=-1).to(torch.bfloat16)

    return {"q": one(s["q"], s["weights"][0]), "k": one(s["k"], s["weights"][1])}


def _plain_store(s):
    # The cache comes back as its bytes: each is defined bit by bit by the arithmetic of the quantisers.
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    cache = s["cache"]
    flat = {n: t.flatten(0, 1) for n, t in cache.items()}

    def int4(x, name):
        x = x[kept].float()
        low, high = x.amin(-1), x.amax(-1)
        scale = _over(high - low, 15.0).to(torch.bfloat16).float()
        scale = torch.where(scale == 0, torch.maximum(low.abs(), high.abs()).to(torch.bfloat16).float(), scale)
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        zero = (torch.round(-low / scale) + 0.0).to(torch.bfloat16).float()
        codes = torch.round(x / scale[..., None] + zero[..., None]).clamp(0, 15).to(torch.uint8)
        flat[name + "_codes"][slots] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        flat[name + "_scales"][slots] = scale.to(torch.bfloat16)
        flat[name + "_zeros"][slots] = zero.to(torch.bfloat16)

    def fp8(x, name):
        scaled = (x[kept].float() / s[name + "_scale"]).clamp(-448, 448)
        flat[name + "_codes"][slots] = scaled.to(torch.float8_e4m3fn).view(torch.uint8)

    put = int4 if s["case"]["form"] == "int4" else fp8
    put(s["k"], "k")
    put(s["v"], "v")
    return cache


def _attend(q, k, v, number):
    """Causal attention of one sequence, [L][heads][D] each, in the type `number`; the scores of as many key heads
    at a time as stay within a few gigabytes."""
    length, heads, dim = q.shape
    group = heads // k.shape[1]
    at_once = max(1, (1 << 31) // max(1, group * length * length))
    later = torch.arange(length, device=q.device)[None] > torch.arange(length, device=q.device)[:, None]

    def some(q, k, v):
        scores = q.to(number) @ k.to(number).unsqueeze(1).transpose(-1, -2) / math.sqrt(dim)
        scores = scores.masked_fill_(later, -math.inf)
        p = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
        return (p @ v.to(number).unsqueeze(1)) / p.sum(-1, keepdim=True)

    q = q.transpose(0, 1).unflatten(0, (-1, group))
    k, v = k.transpose(0, 1), v.transpose(0, 1)
    parts = [some(*t) for t in zip(q.split(at_once), k.split(at_once), v.split(at_once))]
    return torch.cat(parts).flatten(0, 1).transpose(0, 1)


def _plain_attention(s):
    out = [_attend(s["q"][a:b], s["k"][a:b], s["v"][a:b], torch.float32).to(torch.bfloat16)
           for a, b in s["spans"] if b > a]
    return torch.cat(out)


_PLAIN = {"quantize_tokens": _plain_quantize_tokens, "matmul": _plain_matmul, "norm_rope": _plain_norm_rope,
          "store": _plain_store, "attention": _plain_attention}


# --------------------------------------------------------------------------------------------------------------
# The framework's calls
# --------------------------------------------------------------------------------------------------------------

def _own_run(s):
    import group_wise_weight_b200 as wq

    op = s["case"]["op"]
    if op == "quantize_tokens":
        codes, scales = wq.wq_quantize_int8_tokens(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "matmul":
        if "workspace" not in s:  # a program keeps one workspace for its stream
            m, n, k = s["case"]["rows"], s["case"]["outputs"], s["case"]["width"]
            s["workspace"] = torch.zeros(wq.wq_gemm_w8a8_int8_workspace_bytes(m, n, k), dtype=torch.uint8,
                                         device=DEVICE)
        return wq.wq_gemm_w8a8_int8(s["xq"], s["xscales"], s["weight"], s["scales"], workspace=s["workspace"])
    if op == "norm_rope":
        q, k = wq.wq_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["weights"][0],
                                  k_weight=s["weights"][1], eps=1e-6, interleaved=s["case"]["interleaved"])
        return {"q": q, "k": k}
    if op == "store":
        c = s["cache"]
        if s["case"]["form"] == "int4":
            wq.wq_kv_store_int4(s["k"], s["v"], s["slots"], c["k_codes"], c["k_scales"], c["k_zeros"], c["v_codes"],
                                c["v_scales"], c["v_zeros"])
        else:
            wq.wq_kv_store_fp8(s["k"], s["v"], s["slots"], c["k_codes"], s["k_scale"], c["v_codes"], s["v_scale"])
        return c
    return wq.wq_prompt_attention(s["q"], s["k"], s["v"], s["starts"])


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------------------------
# 64-bit references
# --------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize_tokens":
        top = torch.linalg.vector_norm(s["x"].double(), ord=math.inf, dim=1) / 127
        return {"codes": None, "scales": top + (top == 0)}
    if op == "matmul":
        y = torch.einsum("mk,nk->mn", s["xq"].double(), s["weight"].double())
        return torch.einsum("mn,m,n->mn", y, s["xscales"].double(), s["scales"].double())
    if op == "norm_rope":
        half, rotated = case["rotated"] // 2, case["rotated"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                           torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]
        found = {}
        for name, weight in zip(("q", "k"), s["weights"]):
            x = s[name].double().clone()
            if weight is not None:
                power = torch.linalg.vector_norm(x, dim=-1, keepdim=True).pow(2) / case["dim"]
                x = x / (power + 1e-6).sqrt() * weight.double()
            at = torch.arange(half, device=DEVICE)
            first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            found[name] = x
        return found
    if op == "store":
        if case["form"] != "int4":
            return None
        found = {"k_codes": None, "v_codes": None}
        rows = torch.nonzero(s["slots"] >= 0).flatten()
        for name in ("k", "v"):
            x = s[name].double()[rows]
            scale = ((x.amax(-1) - x.amin(-1)).float().double() / 15).to(torch.bfloat16).double()
            kept = {"scales": scale, "zeros": torch.round((-x.amin(-1) / scale).float()).to(torch.bfloat16).double()}
            for part, values in kept.items():
                whole = s["cache"][name + "_" + part].double()
                whole.view(-1, case["kv_heads"])[s["slots"][rows]] = values
                found[name + "_" + part] = whole
        return found
    if sum(n * n for n in _lengths(case)) * case["heads"] * case["dim"] > 16384 * 16384 * 64 * 128:
        return None
    found = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    for a, b in s["spans"]:
        for h in range(case["heads"]):  # one head at a time, by log-sum-exp
            j = h // (case["heads"] // case["kv_heads"])
            scores = torch.einsum("id,jd->ij", s["q"][a:b, h].double(), s["k"][a:b, j].double()) * case["dim"] ** -0.5
            scores = torch.where(torch.ones_like(scores, dtype=torch.bool).tril(), scores, -math.inf)
            weights = torch.exp(scores - torch.logsumexp(scores, dim=1, keepdim=True))
            found[a:b, h] = torch.einsum("ij,jd->id", weights, s["v"][a:b, j].double())
    return found
