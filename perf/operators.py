"""Cases of the stand-alone operators around the quantised experts.

Three operators are measured, each the way a program around the expert layer
calls it:

  norm     moe_block_norm: the experts' rows combined by router weight (or one
           branch row per token), normalised, gated, scaled and added to the
           residual stream, and the next block's normalised input, in one pass;
  int8     moe_quantize_rows + moe_int8_matmul: activations quantised to 8 bits
           per token (gathered into expert order on the way), then the integer
           product with one scale per token and one per output channel, dense or
           grouped by expert;
  grouped  moe_grouped_matmul: products of 16-bit experts with ragged row counts.

`run` computes a case in plain torch (32-bit arithmetic, one rounding at the
end) while `own` is false, and through the library's calls while it is true.
`exact` is the operators' definition in 64 bits, written apart from `run`.
Sizes are those of the repository's configurations (d_model 256, 2048, 4096,
7168; d_ff 512, 1408, 2048, 14336; 4 to 256 experts, top-2, 6 and 8).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(T, K, k=0, dtype="bf16", res="bf16", gate="none", post=True, scale=1.0, offset=0.0, name=None):
    """k: routed rows combined per token (0: the branch is one row per token).
    gate: none, channel [K], token (sigmoid of one value per token) or element [T, K]."""
    d = {"op": "norm", "T": T, "K": K, "k": k, "dtype": dtype, "res": res, "gate": gate, "post": post,
         "scale": scale, "offset": offset}
    return dict(d, name=name) if name else d


def _mm(op, T, E, k, K, N, dtype="bf16", out="bf16", zipf=0.0, name=None):
    """k = 0: dense, all T rows through one matrix; k > 0: T tokens routed to k of E experts."""
    d = {"op": op, "T": T, "E": E, "k": k, "K": K, "N": N, "dtype": dtype, "out": out, "zipf": zipf}
    return dict(d, name=name) if name else d


def listed():
    return [
        # one token of a decode step behind a shared expert: latency alone
        _norm(1, 4096, name="norm_one_token"),
        # decode batch of the 256-expert layer: 8 expert rows per token, fp32 residual stream, gated branch
        _norm(128, 7168, k=8, res="fp32", gate="token", scale=2.5, name="norm_combine_decode"),
        # a width that no vector load fits, per-element gate, (1 + w) norms, odd token count
        _norm(1027, 2051, dtype="fp16", res="fp16", gate="element", offset=1.0, name="norm_odd_width"),
        # prefill chunk of the 8-expert layer: bandwidth alone
        _norm(8192, 4096, k=2, gate="channel", scale=0.5, name="norm_combine_prefill"),
        # one token through a shared expert's gate/up: latency and a split along K
        _mm("int8", 1, 1, 0, 2048, 2816, name="int8_one_token"),
        # decode batch over 64 experts with skewed routing: weight streaming
        _mm("int8", 256, 64, 6, 2048, 2816, zipf=1.1, name="int8_decode_64_experts"),
        # a prefill chunk of odd length through a shared expert
        _mm("int8", 4095, 1, 0, 7168, 4096, name="int8_prefill_shared"),
        # the down projection of a large prefill
        _mm("int8", 8192, 8, 2, 14336, 4096, dtype="fp16", out="fp16", name="int8_prefill_down"),
        # one token on the tiny layer: the smallest call
        _mm("grouped", 1, 4, 2, 256, 1024, name="grouped_one_token"),
        # decode batch of the 8-expert layer: 1.9 GB of weights streamed
        _mm("grouped", 64, 8, 2, 4096, 28672, name="grouped_decode"),
        # prefill over 64 experts with skewed routing: ragged rows per expert
        _mm("grouped", 4096, 64, 6, 2048, 2816, dtype="fp16", out="fp32", zipf=1.1, name="grouped_prefill_64_experts"),
        # the down projection of a large prefill: compute alone
        _mm("grouped", 8192, 8, 2, 14336, 4096, name="grouped_prefill_down"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "int8", "grouped"])
    if op == "norm":
        K = _log(rng, 64, 14336)
        if rng.random() < 0.7:
            K = max(8, K // 8 * 8)
        k = rng.choice([0, 0, 2, 6, 8])
        T = min(_log(rng, 1, 16384), max(1, 8192 * 4096 * 5 // (K * (max(k, 1) + 3))))
        dtype = rng.choice(["bf16", "fp16"])
        return _norm(T, K, k, dtype, rng.choice([dtype, "fp32"]), rng.choice(["none", "token", "channel", "element"]),
                     rng.random() < 0.7, rng.choice([1.0, 0.5, 2.5]), rng.choice([0.0, 1.0]))
    step = 16 if op == "int8" else 8
    K = max(step, _log(rng, 64, 14336) // step * step)
    N = _log(rng, 32, 16384)
    if rng.random() < 0.7:
        N = max(16, N // 16 * 16)
    E = rng.choice([1, 4, 8, 16, 64, 256])
    # at most 2 G weights, and no more products than the largest listed case
    E = max(1, min(E, 2_000_000_000 // (N * K)))
    k = 0 if E == 1 else min(E, rng.choice([1, 2, 6, 8]))
    most = max(1, int(8192 * 2 * 14336 * 4096 / (N * K * max(k, 1))))
    T = min(_log(rng, 1, 16384), most)
    dtype = rng.choice(["bf16", "fp16"])
    return _mm(op, T, E, k, K, N, dtype, rng.choice([dtype, "fp32"]), rng.choice([0.0, 1.1]))


def work(case):
    T, K, k = case["T"], case["K"], case["k"]
    if case["op"] == "norm":
        es, rs = SIZE[case["dtype"]], SIZE[case["res"]]
        gate = {"none": 0, "channel": K, "token": T, "element": T * K}[case["gate"]]
        rows = T * max(k, 1)
        nbytes = rows * K * es + 2 * T * K * rs + T * K * es + gate * es + (2 if case["post"] else 1) * K * es
        nbytes += 8 * T * k
        return {"bytes": nbytes, "flops": T * K * (2 * max(k, 1) + 12)}
    E, N = case["E"], case["N"]
    R = T * max(k, 1)
    used = min(E, R)
    out = R * N * SIZE[case["out"]]
    if case["op"] == "int8":
        # activations read once as 16 bits, weights as 8-bit codes with a scale per channel
        return {"bytes": T * K * 2 + used * N * (K + 4) + out + (4 * R if k else 0), "flops": 2 * R * N * K}
    return {"bytes": R * K * 2 + used * N * K * 2 + out, "flops": 2 * R * N * K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(shape, std, dtype, gen):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _route(T, E, k, zipf, gen):
    """Router logits N(0,1) with a Zipf bias over the experts; the selected pairs in expert order."""
    logits = _randn((T, E), 1.0, torch.float32, gen)
    if zipf > 0:
        place = torch.randperm(E, generator=gen, device="cuda")
        logits -= zipf * torch.log(place.float() + 1.0)
    top, idx = torch.topk(logits, k, dim=1)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * k, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0).to(torch.int32)
    return {"weights": torch.softmax(top, dim=1).contiguous(), "offsets": offsets,
            "perm": (order // k).to(torch.int32), "inv": inv.reshape(T, k).to(torch.int32).contiguous()}


def _int8_weights(E, N, K, gen):
    """8-bit codes of N(0, 0.02) weights, one scale per output channel, made one expert at a time."""
    q = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    s = torch.empty((E, N), dtype=torch.float32, device="cuda")
    for e in range(E):
        w = _randn((N, K), 0.02, torch.float32, gen)
        s[e] = w.abs().amax(1) / 127.0
        q[e] = torch.round(w / s[e][:, None]).clamp_(-127, 127).to(torch.int8)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    T, K, k = case["T"], case["K"], case["k"]
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "norm":
        if k:
            r = _route(T, 8 * k, k, 1.1, gen)
            st["inv"], st["pw"] = r["inv"], r["weights"]
        else:
            st["inv"] = st["pw"] = None
        st["y"] = _randn((T * max(k, 1), K), 0.5, dt, gen)
        # a residual stream with a few channels far larger than the rest
        loud = 1.0 + 20.0 * (torch.rand(K, generator=gen, device="cuda") < 0.005).float()
        st["residual"] = (_randn((T, K), 1.0, torch.float32, gen) * loud).to(DTYPES[case["res"]])
        shift = case["offset"]
        st["w_pre"] = (1.0 - shift + _randn((K,), 0.1, torch.float32, gen)).to(dt)
        st["w_post"] = (1.0 - shift + _randn((K,), 0.1, torch.float32, gen)).to(dt) if case["post"] else None
        shape = {"none": None, "channel": (K,), "token": (T, 1), "element": (T, K)}[case["gate"]]
        st["gate"] = None if shape is None else _randn(shape, 1.0, dt, gen)
        return st
    E, N = case["E"], case["N"]
    if k:
        r = _route(T, E, k, case["zipf"], gen)
        st["offsets"], st["perm"] = r["offsets"], r["perm"]
    else:
        st["offsets"] = st["perm"] = None
    if case["op"] == "int8":
        st["x"] = _randn((T, K), 1.0, dt, gen)
        st["wq"], st["ws"] = _int8_weights(E, N, K, gen)
    else:
        st["x"] = _randn((T * max(k, 1), K), 1.0, dt, gen)
        st["w"] = torch.empty((E, N, K), dtype=dt, device="cuda")
        for e in range(E):
            st["w"][e] = _randn((N, K), 0.02, torch.float32, gen)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(st):
    import bit_quantized_moe_top_b200 as bq
    c = st["case"]
    if c["op"] == "norm":
        return bq.moe_block_norm(st["residual"], st["y"], w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gate"],
                                 gate_sigmoid=c["gate"] == "token", branch_scale=c["scale"], eps=EPS,
                                 weight_offset=c["offset"], inv_pos=st["inv"], pair_weights=st["pw"])
    if c["op"] == "int8":
        q, s = bq.moe_quantize_rows(st["x"], st["perm"])
        return bq.moe_int8_matmul(q, s, st["wq"], st["ws"], st["offsets"], out_dtype=DTYPES[c["out"]])
    return bq.moe_grouped_matmul(st["x"], st["w"], st["offsets"], out_dtype=DTYPES[c["out"]])


def _rms(v, w, offset):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * (offset + w.float())


def _plain_norm(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    if c["k"]:
        b = (st["y"][st["inv"].long()].float() * st["pw"][:, :, None]).sum(1)
    else:
        b = st["y"].float()
    if st["w_post"] is not None:
        b = _rms(b, st["w_post"], c["offset"])
    if st["gate"] is not None:
        g = st["gate"].float()
        b = b * (1.0 / (1.0 + torch.exp(-g)) if c["gate"] == "token" else g)
    r = st["residual"].float() + c["scale"] * b
    return r.to(st["residual"].dtype), _rms(r, st["w_pre"], c["offset"]).to(dt)


def _groups(st):
    """(rows, expert) of each expert that has any, from the offsets on the host."""
    if st["offsets"] is None:
        return [(slice(0, None), 0)]
    o = st["offsets"].tolist()
    return [(slice(o[e], o[e + 1]), e) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def _plain_int8(st):
    c = st["case"]
    x = st["x"] if st["perm"] is None else st["x"][st["perm"].long()]
    xf = x.float()
    top = xf.abs().amax(1, keepdim=True)
    q = torch.round(xf * 127.0 / torch.where(top > 0, top, torch.ones_like(top)))
    s = top / 127.0
    y = torch.empty((x.shape[0], c["N"]), dtype=DTYPES[c["out"]], device=x.device)
    for rows, e in _groups(st):
        y[rows] = ((q[rows] @ st["wq"][e].float().t()) * s[rows] * st["ws"][e][None, :]).to(y.dtype)
    return y


def _plain_grouped(st):
    c = st["case"]
    x = st["x"]
    y = torch.empty((x.shape[0], c["N"]), dtype=DTYPES[c["out"]], device=x.device)
    for rows, e in _groups(st):
        y[rows] = (x[rows].float() @ st["w"][e].float().t()).to(y.dtype)
    return y


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "int8": _plain_int8, "grouped": _plain_grouped}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(st):
    c, f8 = st["case"], torch.float64
    T, K = c["T"], c["K"]
    residual, y = st["residual"].to(f8), st["y"].to(f8)
    if c["k"]:
        branch = torch.zeros((T, K), dtype=f8, device=y.device)
        for j in range(c["k"]):
            branch += st["pw"][:, j].to(f8).unsqueeze(1) * y.index_select(0, st["inv"][:, j].long())
    else:
        branch = y
    if st["w_post"] is not None:
        size = torch.sqrt(branch.square().sum(1) / K + EPS)
        branch = branch / size.unsqueeze(1) * (st["w_post"].to(f8) + c["offset"])
    if c["gate"] == "token":
        branch = branch * torch.sigmoid(st["gate"].to(f8))
    elif c["gate"] != "none":
        branch = branch * st["gate"].to(f8)
    stream = residual + c["scale"] * branch
    size = torch.sqrt(stream.square().sum(1) / K + EPS)
    return stream, stream / size.unsqueeze(1) * (st["w_pre"].to(f8) + c["offset"])


def _exact_product(st):
    c, f8 = st["case"], torch.float64
    x = st["x"].to(f8)
    scale = None
    if c["op"] == "int8":
        if st["perm"] is not None:
            x = x.index_select(0, st["perm"].long())
        top = x.abs().max(dim=1).values
        # codes are whole numbers: 127 x / max |x| to the nearest, halves to even
        x = torch.round(127.0 * x / top.clamp_min(1e-300).unsqueeze(1))
        scale = top / 127.0
    y = torch.empty((x.shape[0], c["N"]), dtype=f8, device=x.device)
    edges = [0, x.shape[0]] if st["offsets"] is None else st["offsets"].tolist()
    for e, (a, b) in enumerate(zip(edges[:-1], edges[1:])):
        if a == b:
            continue
        w = st["wq"][e].to(f8) * st["ws"][e].to(f8).unsqueeze(1) if c["op"] == "int8" else st["w"][e].to(f8)
        y[a:b] = torch.matmul(x[a:b], w.transpose(0, 1))
    return y if scale is None else y * scale.unsqueeze(1)


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_norm(st) if case["op"] == "norm" else _exact_product(st)
