"""Low-rank adapters beside a shared projection (forward and backward) and the AdamW step that trains
them: the cases that are measured, their inputs, and the operators in plain torch operations.

  lora_forward   y[t] = base[t] + s_a B_a (A_a x[t]) with a = idx[t]; a token without an adapter
                 (idx -1) keeps base[t]. Several projections of the same tokens go in one call.
  lora_backward  dx[t] = s_a A_a^T (B_a^T dy[t]) summed over the projections that read x,
                 dA_a = s_a sum_t (B_a^T dy[t]) x[t]^T, dB_a = s_a sum_t dy[t] (A_a x[t])^T
  adamw          one AdamW step over many tensors, moments in 32 bits or in 8 bits with a scale for
                 each 256 elements; the gradients' 2-norm clipped first, or a factor given

Adapter a uses the first ranks[a] of the rank rows its pool has; what lies behind them is not read.
The 8-bit moments: exp_avg as e4m3 and exp_avg_sq as an unsigned float of 5 exponent and 3 fraction
bits, each times its block's scale, rounded up or down at random in proportion to the distance. The
random bits are the outputs of splitmix64 for (seed, step, tensor, element), so they are inputs too.
"""
import math

import numpy as np
import torch

own = False  # the tools set it: plain operations where false, the framework's calls where true

# the projections of the decoder-layer configuration of this repository, (rows, cols) = (out, in)
PROJ = {"q": (4096, 3584), "k": (2048, 3584), "v": (2048, 3584), "o": (3584, 4096), "gate": (14336, 3584),
        "up": (14336, 3584), "down": (3584, 14336), "qkv": None, "wide_up": (25600, 5120), "wide_k": (1024, 5120)}
QKV = ("q", "k", "v")
BLOCK = 256


def _lora(name, op, proj, tokens, adapters, rank, ragged, route, none, out):
    """route: "runs" (each adapter's tokens stand together, as in a batch of prompts) or "mixed" (every
    token its own, as in decoding); none: share of tokens in per cent without an adapter; out: y and dx type."""
    return {"name": name, "op": op, "proj": proj, "tokens": tokens, "adapters": adapters, "rank": rank,
            "ragged": ragged, "route": route, "none": none, "out": out}


def _adamw(name, tensors, scale, param, grad, bits, master, step, max_norm):
    """max_norm: what the gradients' norm is clipped to; 0 where the factor is given."""
    return {"name": name, "op": "adamw", "tensors": tensors, "scale": scale, "param": param, "grad": grad, "bits": bits,
            "master": master, "step": step, "max_norm": max_norm}


def listed():
    return [
        # one sequence decoding: q, k and v of a layer, one token; latency is all
        _lora("decode_one_token", "lora_forward", "qkv", 1, 8, 16, False, "mixed", 0, "float32"),
        # a serving batch, every request its own adapter, of different ranks
        _lora("decode_many_adapters", "lora_forward", "gate,up", 37, 24, 64, True, "mixed", 10, "float32"),
        # prompts of several requests
        _lora("prefill_prompts", "lora_forward", "down", 2049, 6, 16, True, "runs", 12, "float32"),
        # a training batch, two adapters, activations in BF16
        _lora("train_forward", "lora_forward", "gate", 8192, 2, 64, False, "runs", 0, "bfloat16"),
        # gradients for a short ragged batch of several adapters: q, k and v read the same x
        _lora("gradients_short", "lora_backward", "qkv", 333, 5, 8, True, "mixed", 8, "float32"),
        # gradients of a training batch
        _lora("gradients_train", "lora_backward", "gate", 8192, 2, 64, False, "runs", 0, "bfloat16"),
        # every adapter matrix of a 42-layer model at rank 16, 588 tensors: the norm, then the step in 32 bits
        _adamw("adamw_adapters", "adapters", 16, "bfloat16", "float32", 32, True, 100, 1.0),
        # a decoder layer trained whole, moments in 32 bits
        _adamw("adamw_layer", "layer", 1, "bfloat16", "bfloat16", 32, False, 3, 1.0),
        # the same with moments in 8 bits, the factor given
        _adamw("adamw_layer_8bit", "layer", 1, "bfloat16", "bfloat16", 8, False, 1000, 0.0),
        # a few small tensors of odd sizes, the first step, in 32 and in 8 bits
        _adamw("adamw_odd", "odd", 7, "float32", "float32", 32, False, 0, 0.5),
        _adamw("adamw_odd_8bit", "odd", 11, "float32", "float32", 8, False, 0, 0.0),
    ]


def draw(rng):
    lg = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    kind = rng.choice(["lora_forward", "lora_forward", "lora_backward", "lora_backward", "adamw", "adamw", "adamw"])
    if kind.startswith("lora"):
        tokens = lg(1, 6000)
        proj = rng.choice(["qkv", "q", "o", "gate", "down", "gate,up", "wide_k"])
        return _lora("drawn", kind, proj, tokens, min(lg(1, 40), max(1, 65536 // tokens)), rng.choice([8, 16, 24, 32, 64, 72, 128]),
                     rng.random() < 0.5, rng.choice(["runs", "mixed"]), rng.choice([0, 0, 15, 60]),
                     rng.choice(["float32", "bfloat16"])) | {"name": "drawn_%d" % rng.randrange(1 << 30)}
    tensors = rng.choice(["odd", "adapters"])
    scale = lg(1, 400) if tensors == "odd" else rng.choice([1, 2, 3, 5, 8, 12])
    param, bits = rng.choice(["float32", "bfloat16"]), rng.choice([8, 32])
    return _adamw("drawn_%d" % rng.randrange(1 << 30), tensors, scale, param, rng.choice(["float32", "bfloat16"]), bits,
                  param == "bfloat16" and rng.random() < 0.5, rng.choice([0, 1, 17, 5000]),
                  rng.choice([0.0, 0.5, 1000.0]) if bits == 32 else 0.0)


# ------------------------------------------------------------------------------ sizes of a case
def _projs(case):
    names = QKV if case["proj"] == "qkv" else tuple(case["proj"].split(","))
    return [PROJ[n] for n in names]


def _ranks(case):
    r = case["rank"]
    return [max(1, r - (5 * a) % r) if case["ragged"] else r for a in range(case["adapters"])]


def _tensor_sizes(case):
    """Element counts and weight decays of the tensors of an optimiser case."""
    if case["tensors"] == "layer":
        return [PROJ[p][0] * PROJ[p][1] for p in ("q", "k", "v", "o", "gate", "up", "down")] + [3584] * 4, [0.1] * 7 + [0.0] * 4
    if case["tensors"] == "adapters":
        one = [case["scale"] * d for p in ("q", "k", "v", "o", "gate", "up", "down") for d in PROJ[p]]
        return one * 42, [0.01] * (42 * len(one))
    sizes = [1, 255, 256, 257, 1000 * case["scale"] + 1, 4097, 8 * case["scale"], 3584, 511 * case["scale"]]
    return sizes, [0.0, 0.1, 0.0, 0.1, 0.01, 0.1, 0.0, 0.0, 0.1]


def _used(case):
    """(tokens with an adapter, adapters in use) as the route gives them on average."""
    t, n = case["tokens"], case["adapters"]
    live = t - (t * case["none"]) // 100
    used = n * (1 - (1 - 1 / n) ** live) if case["route"] == "mixed" else min(n, live)
    return live, max(1.0, used) if live else 0.0


def work(case):
    """Bytes that have to be read once and written once, and operations, of one pass."""
    if case["op"] in ("lora_forward", "lora_backward"):
        t, out = case["tokens"], 4 if case["out"] == "float32" else 2
        live, used = _used(case)
        ranks = _ranks(case)
        r = sum(ranks) / len(ranks)
        projs = _projs(case)
        weights = sum(2 * used * r * (n + k) for n, k in projs)
        flops = sum(2 * live * r * (n + k) for n, k in projs)
        x = 2 * live * projs[0][1]
        if case["op"] == "lora_forward":
            return {"bytes": x + weights + sum(2 * out * t * n for n, _ in projs), "flops": flops}
        grads = sum(4 * case["adapters"] * case["rank"] * (n + k) for n, k in projs)
        return {"bytes": x + weights + sum(2 * live * n for n, _ in projs) + grads + out * t * projs[0][1], "flops": 3 * flops}
    n = sum(_tensor_sizes(case)[0])
    g = 4 if case["grad"] == "float32" else 2
    p = 4 if case["param"] == "float32" else 2
    if case["bits"] == 8:  # codes in and out, and the values they stand for, which are returned
        state = 2 * (1 + 1 + 4) + 8 / BLOCK * 2
    else:
        state = 16
    norm = g if case["max_norm"] else 0  # no gradient is used before the norm of all is known
    return {"bytes": n * (norm + g + (p + 8 if case["master"] else 2 * p) + state), "flops": 15 * n}


# ------------------------------------------------------------------------------ inputs
def _type(name):
    return getattr(torch, name)


def _lora_inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    nrm = lambda shape, scale, dt: (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)  # noqa: E731
    t, n, r = case["tokens"], case["adapters"], case["rank"]
    projs, bf = _projs(case), torch.bfloat16
    if case["route"] == "mixed":
        idx = torch.randint(0, n, (t,), generator=gen, device="cuda", dtype=torch.int32)
        drop = torch.randperm(t, generator=gen, device="cuda")[: (t * case["none"]) // 100]
    else:  # runs of uneven length, the tokens without an adapter at the end, as padding is
        live = t - (t * case["none"]) // 100
        cut = [live * (2 * a + a * a) // (2 * n + n * n) for a in range(n + 1)]
        idx = torch.repeat_interleave(torch.arange(n, device="cuda", dtype=torch.int32),
                                      torch.tensor([cut[a + 1] - cut[a] for a in range(n)], device="cuda"))
        idx = torch.cat([idx, idx.new_zeros(t - live)])
        drop = torch.arange(live, t, device="cuda")
    idx[drop] = -1
    s = {"op": case["op"], "out": _type(case["out"]), "idx": idx, "r": r, "n": n,
         "ranks": torch.tensor(_ranks(case), device="cuda", dtype=torch.int32),
         "scales": torch.rand(n, generator=gen, device="cuda") + 0.5,
         "x": nrm((t, projs[0][1]), 1.0, bf),
         "a": [nrm((n, r, k), k ** -0.5, bf) for _, k in projs],
         "b": [nrm((n, m, r), r ** -0.5, bf) for m, _ in projs]}
    if case["op"] == "lora_forward":
        s["base"] = [nrm((t, m), 1.0, s["out"]) for m, _ in projs]
    else:
        s["dy"] = [nrm((t, m), 0.1, bf) for m, _ in projs]
    return s


def _adamw_inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    sizes, decay = _tensor_sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]  # every tensor starts on a block of its own in the flat buffers
    total = BLOCK * sum(blocks)
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    s = {"op": case["op"], "sizes": sizes, "decay": decay, "starts": [BLOCK * sum(blocks[:k]) for k in range(len(sizes))]}
    for n, at in zip(sizes, s["starts"]):
        live[at:at + n] = True
    grad = torch.randn(total, generator=gen, device="cuda") * 0.01
    s["grad"] = torch.where(live, grad, 0).to(_type(case["grad"]))
    del grad
    param = torch.where(live, torch.randn(total, generator=gen, device="cuda") * 0.02, 0)
    m = torch.where(live, torch.randn(total, generator=gen, device="cuda") * 0.003, 0)
    v = torch.where(live, (torch.randn(total, generator=gen, device="cuda") * 0.01).square_(), 0)
    if case["step"] == 0:
        m.zero_()
        v.zero_()
    s |= {"param": param.to(_type(case["param"])), "master": param if case["master"] else None, "bits": case["bits"],
          "lr": 1e-3, "clip": 0.75, "max_norm": case["max_norm"], "step": case["step"], "betas": (0.9, 0.999), "eps": 1e-8, "seed": 17}
    if case["bits"] == 32:
        s |= {"m": m, "v": v}
    else:  # codes of any kind are a valid state: signs and magnitudes drawn, padding zero
        zero = 0 if case["step"] == 0 else 1
        mc = torch.randint(0, 256, (total,), generator=gen, device="cuda", dtype=torch.uint8)
        mc = torch.where((mc & 127) == 127, mc - 1, mc)
        vc = torch.randint(150, 0xF8, (total,), generator=gen, device="cuda", dtype=torch.uint8)
        s |= {"mc": torch.where(live, mc, 0) * zero, "vc": torch.where(live, vc, 0) * zero,
              "ms": m.view(-1, BLOCK).abs().amax(1) / 448, "vs": v.view(-1, BLOCK).amax(1) / 61440}
    if not own:  # per block: weight decay, number of the tensor, first element
        at = torch.tensor(blocks, device="cuda")
        rep = lambda v, dt: torch.repeat_interleave(torch.tensor(v, device="cuda", dtype=dt), at)  # noqa: E731
        s |= {"b_decay": rep(decay, torch.float32)[:, None], "b_tensor": rep(list(range(len(sizes))), torch.int64)[:, None]}
        s["b_first"] = (torch.arange(sum(blocks), device="cuda") * BLOCK - rep(s["starts"], torch.int64))[:, None]
    return s


def prepare(case, seed):
    if case["op"].startswith("lora"):
        s = _lora_inputs(case, seed)
        if own:  # what a program keeps: the adapter set, the batch's routing and its buffers
            import lossless_entropy_coding_interleaved_b200 as bs
            t = case["tokens"]
            s["set"] = bs.LoraAdapters(s["a"], s["b"], s["scales"], s["ranks"])
            s["plan"] = bs.LoraPlan(t, s["n"], device="cuda")
            s["state"] = s["set"].state(t)
            if case["op"] == "lora_forward":
                s["y"] = [torch.empty_like(b) for b in s["base"]]
            else:
                s["work"] = s["set"].state(t)
                s["dx"] = torch.empty(s["x"].shape, dtype=s["out"], device="cuda")
                s["da"] = [torch.empty(a.shape, dtype=torch.float32, device="cuda") for a in s["a"]]
                s["db"] = [torch.empty(b.shape, dtype=torch.float32, device="cuda") for b in s["b"]]
                # the forward pass left A x behind for the backward pass
                s["plan"].update(s["idx"])
                s["set"].forward(s["plan"], [s["x"]] * len(s["a"]), None, state=s["state"])
        return s
    s = _adamw_inputs(case, seed)
    if own:
        import lossless_entropy_coding_interleaved_b200 as bs
        cut = lambda flat: [flat[at:at + n] for n, at in zip(s["sizes"], s["starts"])]  # noqa: E731
        states = ((cut(s["m"]), cut(s["v"])) if s["bits"] == 32 else
                  tuple([cut(s[c]), [s[f][at // BLOCK: at // BLOCK + -(-n // BLOCK)] for n, at in zip(s["sizes"], s["starts"])]]
                        for c, f in (("mc", "ms"), ("vc", "vs"))))
        s["opt"] = bs.AdamW(cut(s["param"]), cut(s["grad"]), lr=s["lr"], betas=s["betas"], eps=s["eps"], weight_decay=s["decay"],
                            bits=s["bits"], masters=cut(s["master"]) if s["master"] is not None else None, seed=s["seed"],
                            step=s["step"], clip=s["clip"], states=states)
        # a pass leaves the state as it was and writes another one, as a program does that codes the
        # weights of this step while the next one runs
        like = lambda flat: None if flat is None else torch.zeros_like(flat)  # noqa: E731
        s["new"] = {k: like(s.get(k)) for k in ("param", "master", "m", "v", "mc", "vc", "ms", "vs")}
        into = ((cut(s["new"]["m"]), cut(s["new"]["v"])) if s["bits"] == 32 else
                tuple([cut(s["new"][c]), [s["new"][f][at // BLOCK: at // BLOCK + -(-n // BLOCK)] for n, at in zip(s["sizes"], s["starts"])]]
                      for c, f in (("mc", "ms"), ("vc", "vs"))))
        s["twin"] = s["opt"].twin(cut(s["new"]["param"]), cut(s["new"]["master"]) if s["master"] is not None else None, into)
        if s["bits"] == 8:
            s["read"] = [torch.zeros(s["grad"].numel(), device="cuda") for _ in range(2)]
            s["read_cut"] = [cut(f) for f in s["read"]]
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "lora_forward":
        return _forward_plain(s)
    if s["op"] == "lora_backward":
        return _backward_plain(s)
    return _adamw_plain(s)


def _run_own(s):
    if s["op"] == "lora_forward":
        s["plan"].update(s["idx"])
        s["set"].forward(s["plan"], [s["x"]] * len(s["y"]), s["y"], bases=s["base"], state=s["state"])
        return s["y"]
    if s["op"] == "lora_backward":
        k = len(s["a"])
        s["set"].backward(s["plan"], [s["x"]] * k, s["dy"], s["state"], s["da"], s["db"], dxs=[s["dx"]] * k, work=s["work"])
        return {"dx": s["dx"], "da": s["da"], "db": s["db"]}
    s["opt"].step(max_norm=s["max_norm"] or None, into=s["twin"], number=s["step"] + 1)
    out = {"param": s["new"]["param"]}
    if s["max_norm"]:
        out["norm"] = s["opt"].norm
    if s["master"] is not None:
        out["master"] = s["new"]["master"]
    if s["bits"] == 32:
        return out | {"m": s["new"]["m"], "v": s["new"]["v"]}
    s["twin"].read_states(*s["read_cut"])
    return out | {"m": s["read"][0], "v": s["read"][1]}


def _select(s):
    """[tokens, adapters * rank]: whether the token uses that rank row of that adapter."""
    row = torch.arange(s["n"] * s["r"], device="cuda")
    return (s["idx"].long()[:, None] == (row // s["r"])[None]) & ((row % s["r"]) < s["ranks"].long()[row // s["r"]])[None]


def _flat_pools(s, k):
    """A of every adapter as [adapters * rank, cols] and B as [rows, adapters * rank], in 32 bits."""
    n, r = s["n"], s["r"]
    a = s["a"][k].float().reshape(n * r, -1)
    b = s["b"][k].float().permute(1, 0, 2).reshape(-1, n * r)
    return a, b


def _forward_plain(s):
    on, scale = _select(s), torch.repeat_interleave(s["scales"], s["r"])
    x, out = s["x"].float(), []
    for k in range(len(s["a"])):
        a, b = _flat_pools(s, k)
        h = torch.where(on, x @ a.T * scale, 0)
        out.append((s["base"][k].float() + h @ b.T).to(s["out"]))
    return out


def _backward_plain(s):
    on, scale = _select(s), torch.repeat_interleave(s["scales"], s["r"])
    n, r = s["n"], s["r"]
    x, dx, da, db = s["x"].float(), 0, [], []
    for k in range(len(s["a"])):
        a, b = _flat_pools(s, k)
        dy = s["dy"][k].float()
        h = torch.where(on, x @ a.T * scale, 0)
        g = torch.where(on, dy @ b * scale, 0)
        dx = dx + g @ a
        da.append((g.T @ x).reshape(n, r, -1))
        db.append((dy.T @ h).reshape(-1, n, r).permute(1, 0, 2))
    return {"dx": dx.to(s["out"]), "da": da, "db": db}


# The 8-bit floats by their definition: (8 + f) 2^(e - bias - 3), or f 2^(1 - bias - 3) for e = 0.
def _table(bias, size):
    c = np.arange(size)
    return ((c & 7) + np.where(c >> 3, 8, 0)) * 2.0 ** (np.maximum(c >> 3, 1) - bias - 3)


def _values(table, codes):
    return torch.tensor(table, dtype=torch.float32, device="cuda")[codes.long()]


def _decode_e4m3(c):
    return _values(np.concatenate([_table(7, 128), -_table(7, 128)]), c)


def _decode_u53(c):
    return _values(_table(15, 256), c)


def _code(y, u, bias, most):
    """Codes of y >= 0 (float32), rounded up where the 16 random bits u reach the rest: floor(y / q + u / 2^16) q."""
    small = (y * 2.0 ** (bias + 2) + u.float() * 2.0 ** -16).int()
    normal = ((y.view(torch.int32) + (u << 4)) >> 20) - ((127 - bias) << 3)
    return torch.clamp(torch.where(y < 2.0 ** (1 - bias), small, normal), max=most)


def _shift(z, k):
    return (z >> k) & ((1 << (64 - k)) - 1)


def _i64(v):
    return v - (1 << 64) if v >= 1 << 63 else v


GOLDEN, MIX1, MIX2 = _i64(0x9E3779B97F4A7C15), _i64(0xBF58476D1CE4E5B9), _i64(0x94D049BB133111EB)


def _mix(z):
    """The output function of splitmix64, on 64-bit integers that wrap."""
    z = (z ^ _shift(z, 30)) * MIX1
    z = (z ^ _shift(z, 27)) * MIX2
    return z ^ _shift(z, 31)


def _random_bits(s):
    """Two lots of 16 random bits for every element, from one 64-bit output for each pair of elements."""
    key = _mix(_mix(torch.full_like(s["b_tensor"], s["seed"]) + (s["step"] + 1) * 2654435769) + s["b_tensor"])
    e = s["b_first"] + torch.arange(BLOCK, device="cuda")
    z = _mix(key + GOLDEN * ((e >> 1) + 1))
    half = torch.where((e & 1) == 0, z & 0xFFFFFFFF, _shift(z, 32)).to(torch.int64)
    return (half & 0xFFFF).int(), (half >> 16).int()


def _quantise(value, top, bias, most, u):
    big = value.abs().amax(1, keepdim=True)
    dead = big < 2.0 ** -100  # a block too small to count
    top = torch.full_like(big, top)
    inv = torch.where(dead, 0, top / big)  # a tensor over a tensor: rounded once
    scale = torch.where(dead, 0, big / top)
    return _code(value.abs() * inv, u, bias, most), scale


def _adamw_plain(s):
    b1, b2 = s["betas"]
    t = s["step"] + 1
    shape = (-1, BLOCK)
    g, clip = s["grad"].float().view(shape), s["clip"]
    if s["max_norm"]:
        norm = g.square().sum(1).double().sum().sqrt()  # the long sum in 64 bits
        clip = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
    g = g * clip
    p = (s["master"] if s["master"] is not None else s["param"].float()).view(shape)
    if s["bits"] == 32:
        m, v = s["m"].view(shape), s["v"].view(shape)
    else:
        m = _decode_e4m3(s["mc"]).view(shape) * s["ms"][:, None]
        v = _decode_u53(s["vc"]).view(shape) * s["vs"][:, None]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * (1 - b2) * g
    step = s["lr"] / (1 - b1 ** t) * m / (torch.sqrt(v) / math.sqrt(1 - b2 ** t) + s["eps"])
    p = p - p * (s["lr"] * s["b_decay"]) - step
    out = {"param": p.view(-1).to(s["param"].dtype)}
    if s["master"] is not None:
        out["master"] = p.view(-1)
    if s["max_norm"]:
        out["norm"] = norm.float()
    if s["bits"] == 32:
        return out | {"m": m.view(-1), "v": v.view(-1)}
    um, uv = _random_bits(s)
    cm, sm = _quantise(m, 448.0, 7, 0x7E, um)
    cv, sv = _quantise(v, 61440.0, 15, 0xF7, uv)
    cv = torch.where((v > 0) & (sv > 0), torch.clamp(cv, min=1), cv)  # what is above zero stays above it
    return out | {"m": (torch.copysign(_decode_e4m3(cm), m) * sm).view(-1), "v": (_decode_u53(cv) * sv).view(-1)}


# ------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    if case["op"].startswith("lora"):
        return _lora_exact(case, _lora_inputs(case, seed))
    return _adamw_exact(_adamw_inputs(case, seed))


def _lora_exact(case, s):
    """One adapter after the other, the tokens it has, in float64."""
    t, ranks = case["tokens"], _ranks(case)
    rows = [torch.nonzero(s["idx"] == a).flatten() for a in range(s["n"])]
    x = s["x"].double()
    ys, das, dbs, dx = [], [], [], torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for k in range(len(s["a"])):
        if case["op"] == "lora_forward":
            y = s["base"][k].double()
        else:
            da = torch.zeros(s["a"][k].shape, dtype=torch.float64, device="cuda")
            db = torch.zeros(s["b"][k].shape, dtype=torch.float64, device="cuda")
        for a, at in enumerate(rows):
            if at.numel() == 0:
                continue
            A, B, c = s["a"][k][a, : ranks[a]].double(), s["b"][k][a, :, : ranks[a]].double(), s["scales"][a].double()
            xa = x[at]
            h = torch.einsum("tk,rk->tr", xa, A) * c
            if case["op"] == "lora_forward":
                y[at] += torch.einsum("tr,nr->tn", h, B)
                continue
            dy = s["dy"][k][at].double()
            g = torch.einsum("tn,nr->tr", dy, B) * c
            dx[at] += torch.einsum("tr,rk->tk", g, A)
            da[a, : ranks[a]] = torch.einsum("tr,tk->rk", g, xa)
            db[a, :, : ranks[a]] = torch.einsum("tn,tr->nr", dy, h)
        if case["op"] == "lora_forward":
            ys.append(y)
        else:
            das.append(da)
            dbs.append(db)
    return ys if case["op"] == "lora_forward" else {"dx": dx, "da": das, "db": dbs}


def _adamw_exact(s):
    """Element after element as numpy has them, 64 bits throughout; up to 60 million elements, or 4 million in 8 bits."""
    if s["grad"].numel() > (60_000_000 if s["bits"] == 32 else 4_000_000):
        return None
    b1, b2 = s["betas"]
    t = s["step"] + 1
    host = lambda v: v.double().cpu().numpy()  # noqa: E731
    start = host(s["master"] if s["master"] is not None else s["param"])
    grad = host(s["grad"])
    norm = float(np.sqrt(np.dot(grad, grad)))
    grad *= min(1.0, s["max_norm"] / (norm + 1e-6)) if s["max_norm"] else s["clip"]
    if s["bits"] == 32:
        m0, v0 = host(s["m"]), host(s["v"])
    else:
        grid = lambda bias, most: np.array([(1 + (c % 8) / 8) * 2.0 ** (c // 8 - bias) if c >= 8 else c * 2.0 ** (-2 - bias)  # noqa: E731
                                            for c in range(most + 1)])
        e4, u5 = grid(7, 127), grid(15, 255)
        mc, vc = s["mc"].cpu().numpy(), s["vc"].cpu().numpy()
        m0 = np.where(mc & 128, -1.0, 1.0) * e4[mc & 127] * np.repeat(host(s["ms"]), BLOCK)
        v0 = u5[vc] * np.repeat(host(s["vs"]), BLOCK)
    m1, v1 = b1 * m0 + (1 - b1) * grad, b2 * v0 + (1 - b2) * grad ** 2
    decay = np.zeros(start.size)
    for n, at, d in zip(s["sizes"], s["starts"], s["decay"]):
        decay[at:at + n] = d
    new = start * (1 - s["lr"] * decay) - s["lr"] * (m1 / (1 - b1 ** t)) / (np.sqrt(v1 / (1 - b2 ** t)) + s["eps"])
    out = {"param": new}
    if s["master"] is not None:
        out["master"] = new
    if s["max_norm"]:
        out["norm"] = np.float64(norm)
    if s["bits"] == 32:
        return out | {"m": m1, "v": v1}
    wrap = (1 << 64) - 1

    def mix(z):
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))

    qm, qv = np.zeros_like(m1), np.zeros_like(v1)
    for number, (n, at) in enumerate(zip(s["sizes"], s["starts"])):
        key = mix(np.array([(s["seed"] + t * 2654435769) & wrap], np.uint64))
        key = mix(key + np.uint64(number))
        z = mix(key + np.uint64(0x9E3779B97F4A7C15) * (np.arange((n + 1) // 2, dtype=np.uint64) + np.uint64(1)))
        half = np.stack([z & np.uint64(0xFFFFFFFF), z >> np.uint64(32)], 1).reshape(-1)[:n]
        um, uv = (half & np.uint64(0xFFFF)).astype(np.float64) / 65536, (half >> np.uint64(16)).astype(np.float64) / 65536
        for value, u, steps, top, out_q, keep in ((m1, um, e4, 448.0, qm, False), (v1, uv, u5, 61440.0, qv, True)):
            x = value[at:at + n]
            pad = np.zeros(-(-n // BLOCK) * BLOCK)
            pad[:n] = np.abs(x)
            scale = np.repeat(pad.reshape(-1, BLOCK).max(1) / top, BLOCK)[:n]
            live = scale * top >= 2.0 ** -100
            y = np.where(live, np.abs(x) / np.where(live, scale, 1.0), 0.0)
            y = np.minimum(y, top)
            low = np.searchsorted(steps[: 0x7F if top == 448.0 else 0xF8], y, side="right") - 1
            high = np.minimum(low + 1, 0x7E if top == 448.0 else 0xF7)
            gap = np.where(high > low, steps[high] - steps[low], 1.0)
            pick = np.where(u + (y - steps[low]) / gap >= 1.0, high, low)
            if keep:
                pick = np.where((x > 0) & live & (pick == 0), 1, pick)
            out_q[at:at + n] = np.sign(x) * steps[pick] * np.where(live, scale, 0.0)
    return out | {"m": qm, "v": qv}
