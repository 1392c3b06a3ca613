"""Cases that measure the operators around the vocabulary layer: 4-bit packing
and the product of two 4-bit matrices (a layer that is only read: the serving
head, a teacher), the next token drawn from the logits, and the loss against a
teacher's top logits with its gradient.

4-bit format: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two
to a byte, the earlier element in the low half, and one power-of-two scale (a
byte b stands for 2^(b-127)) for each 32 elements of a row. The scale bytes lie
in tiles of 128 rows by 128 elements, 512 bytes each, tile row after tile row:
row r's byte for block j is byte (r%32)*16 + (r%128)//32*4 + j%4 of its tile;
bytes of rows and blocks past the end are 127.

With own = False the operators run in plain torch operations; with own = True
through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
B = 32

# The framework's own layers: the large language model's softmax layer
# (267,735 x 1024) and the embedding workload's (33,278 x 512).
LM_ROWS, LM_COLS = 267735, 1024
EMB_ROWS, EMB_COLS = 33278, 512


def listed():
    return [
        # one token's hidden state packed before a serving product (and read back): latency
        {"name": "quant_token", "op": "quant", "rows": 1, "cols": LM_COLS, "dtype": "bf16"},
        # a float32 layer's weight packed for serving, and its values for measuring what the packing cost
        {"name": "quant_weight", "op": "quant", "rows": EMB_ROWS, "cols": EMB_COLS, "dtype": "f32"},
        # the same for the large vocabulary, from a bfloat16 checkpoint
        {"name": "quant_large_weight", "op": "quant", "rows": LM_ROWS, "cols": LM_COLS, "dtype": "bf16"},
        # one token through a square layer: latency, and reading the weight
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16"},
        # a few sequences' next-token logits over the large vocabulary, in float32
        {"name": "matmul_serving_head", "op": "matmul", "m": 24, "n": LM_ROWS, "k": LM_COLS, "dtype": "f32"},
        # a teacher's hidden layer over a training batch
        {"name": "matmul_layer", "op": "matmul", "m": 8192, "n": 4096, "k": 4096, "dtype": "bf16"},
        # one sequence's next token over the small vocabulary: latency
        {"name": "sample_token", "op": "sample", "t": 1, "v": EMB_ROWS, "dtype": "bf16", "mode": "nucleus"},
        # a few sequences' next tokens, each request with its own settings
        {"name": "sample_serving", "op": "sample", "t": 24, "v": LM_ROWS, "dtype": "f32", "mode": "mixed"},
        # a large serving batch
        {"name": "sample_batch", "op": "sample", "t": 256, "v": LM_ROWS, "dtype": "f32", "mode": "mixed"},
        # a small student's step: loss and gradient in float32
        {"name": "distill_small", "op": "distill", "t": 200, "v": EMB_ROWS, "k": 32, "dtype": "f32", "grad": "f32", "hard": False},
        # the loss alone, over an evaluation batch, with the words that followed
        {"name": "distill_eval", "op": "distill", "t": 2048, "v": EMB_ROWS, "k": 100, "dtype": "bf16", "grad": "", "hard": True},
        # a training step over the large vocabulary (odd row length), padded rows among them
        {"name": "distill_train", "op": "distill", "t": 2048, "v": LM_ROWS, "k": 64, "dtype": "bf16", "grad": "bf16", "hard": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "matmul", "matmul", "sample", "sample", "distill", "distill"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "quant":
        rows, cols = _log(rng, 1, LM_ROWS), _log(rng, 32, 8192)
        while rows * cols > LM_ROWS * LM_COLS // 2:
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype}
    if op == "matmul":
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, LM_ROWS), _log(rng, 64, 4096)
        if rng.random() < 0.5:  # half of the widths are multiples of 8, as layers mostly have
            n, k = -(-n // 8) * 8, -(-k // 8) * 8
        while m * n * k > 8192 * 4096 * 4096 or m * n > 1 << 28:
            n = max(64, n // 2)
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype}
    if op == "sample":
        mode = rng.choice(["nucleus", "mixed", "mixed", "plain"])
        return {"op": op, "t": _log(rng, 1, 200), "v": _log(rng, 1000, LM_ROWS), "dtype": dtype, "mode": mode}
    t, v = _log(rng, 1, 2048), _log(rng, 1000, LM_ROWS)
    if rng.random() < 0.5:
        v = -(-v // 8) * 8
    while t * v > 1024 * LM_ROWS:
        t //= 2
    return {"op": op, "t": t, "v": v, "k": _log(rng, 1, 256), "dtype": dtype, "grad": rng.choice(["bf16", "f32", dtype, ""]),
            "hard": rng.random() < 0.5}


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _up(x, y):
    return -(-x // y)


# ---- 4-bit packing, plainly ----

_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(b):
    """2^(b-127) of each byte, from the bits of a float32 (1 <= b <= 254)."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _plain_quant(x):
    """float32 values that the packed x stands for, its codes [rows, blocks of 32] as small integers, and the scale byte of each block."""
    rows, cols = x.shape
    nb = _up(cols, B)
    v = torch.nn.functional.pad(x.float(), (0, nb * B - cols)).reshape(rows, nb, B)
    m, ex = torch.frexp(v.abs().amax(dim=2, keepdim=True))
    # the least e with amax <= 6 * 2^e = 0.75 * 2^(3+e), not below -125
    e = torch.where(m == 0, torch.full_like(ex, -125), (ex - 3 + (m > 0.75)).clamp(min=-125))
    q = v * _pow2(127 - e)
    a = q.abs()
    # to the nearest value; halfway, to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    mag = torch.tensor(_VALUES, device=x.device)[c.int()]
    val = torch.copysign(mag, q) * _pow2(e + 127)
    code = c + 8 * torch.signbit(q).to(torch.uint8)
    return val.reshape(rows, nb * B)[:, :cols], code.reshape(rows, nb * B), (e + 127).to(torch.uint8).reshape(rows, nb)


def _tiled(s, cols):
    """Scale bytes [rows, blocks] in their tiles of 128 x 128 elements."""
    rows, nb = s.shape
    tr, tc = _up(rows, 128), _up(cols, 128)
    p = torch.nn.functional.pad(s, (0, tc * 4 - nb, 0, tr * 128 - rows), value=127)
    return p.reshape(tr, 4, 32, tc, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(s, rows, cols):
    tr, tc = _up(rows, 128), _up(cols, 128)
    return s.reshape(tr, tc, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tr * 128, tc * 4)[:rows, :_up(cols, B)]


def _plain_values(codes, scales, cols):
    """The float32 values of a packed matrix."""
    rows = codes.shape[0]
    pair = torch.stack((codes & 15, codes >> 4), dim=2).reshape(rows, -1)[:, :cols].int()
    v = torch.tensor(_VALUES + tuple(-x for x in _VALUES), device=codes.device)[pair]
    return v * _pow2(_untiled(scales, rows, cols)).repeat_interleave(B, 1)[:, :cols]


def _room(rows, cols):
    """Uninitialised code bytes of a [rows, cols] matrix whose rows start on 16 bytes, and its scale bytes."""
    codes = torch.empty((rows, _up(cols, B) * 16), dtype=torch.uint8, device=DEV)[:, :_up(cols, 2)]
    return codes, torch.empty(_up(rows, 128) * _up(cols, 128) * 512, dtype=torch.uint8, device=DEV)


def _packed(x):
    """x as a user holds it packed."""
    rows, cols = x.shape
    _, code, s = _plain_quant(x)
    code = code.reshape(rows, -1, 2)
    codes, scales = _room(rows, cols)
    codes.copy_((code[:, :, 0] + 16 * code[:, :, 1])[:, :codes.shape[1]])
    scales.copy_(_tiled(s, cols))
    return codes, scales


def _activations(g, rows, cols):
    """Hidden states: unit normal, a few channels and tokens far larger, some tokens zero (padding)."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((1, cols), generator=g, device=DEV))
    x *= 1 + 30 * (torch.rand((1, cols), generator=g, device=DEV) < 0.005)
    if rows > 8:
        x *= torch.rand((rows, 1), generator=g, device=DEV) > 0.02
    return x


def _logits(g, rows, vocab):
    """Next-word logits: a Zipf prior over the words in some order, noise, and a few words that the context makes likely."""
    order = torch.randperm(vocab, generator=g, device=DEV)
    z = torch.randn((rows, vocab), generator=g, device=DEV).mul_(1.2)
    z -= 1.1 * torch.log(1.0 + order)
    likely = torch.randint(vocab, (rows, 12), generator=g, device=DEV)
    z.scatter_add_(1, likely, 6.0 + 2.0 * torch.randn((rows, 12), generator=g, device=DEV))
    return z


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"case": case, "op": case["op"]}
    if case["op"] == "quant":
        rows, cols = case["rows"], case["cols"]
        x = _activations(g, rows, cols) if rows < 8192 else torch.randn((rows, cols), generator=g, device=DEV) * cols ** -0.5
        st["x"] = x.to(_dtype(case["dtype"]))
        st["codes"], st["scales"] = _room(rows, cols)
        st["out"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"], st["xs"] = _packed(_activations(g, m, k))
        st["w"], st["ws"] = _packed(torch.randn((n, k), generator=g, device=DEV) * k ** -0.5)
        st["out"] = torch.empty((m, n), dtype=_dtype(case["dtype"]), device=DEV)
    elif case["op"] == "sample":
        t, v, mode = case["t"], case["v"], case["mode"]
        st["logits"] = _logits(g, t, v).to(_dtype(case["dtype"]))

        def pick(choices):
            return torch.tensor(choices, device=DEV)[torch.randint(len(choices), (t,), generator=g, device=DEV)]

        st["u"] = torch.rand(t, generator=g, device=DEV)
        one = torch.ones(t, device=DEV)
        if mode == "mixed":  # every request has its own; 0 temperature: the likeliest word
            st["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3])
            st["top_k"] = pick([0, 0, 1, 20, 50, 1000]).to(torch.int32)
            st["top_p"] = pick([1.0, 1.0, 0.8, 0.9, 0.95])
            st["min_p"] = pick([0.0, 0.0, 0.02, 0.1])
        else:
            st["temperature"] = one * (0.9 if mode == "nucleus" else 1.0)
            st["top_k"] = st["min_p"] = None
            st["top_p"] = one * 0.92 if mode == "nucleus" else None
        st["tokens"] = torch.empty(t, dtype=torch.int32, device=DEV)
    else:
        t, v, k = case["t"], case["v"], case["k"]
        z = _logits(g, t, v)
        st["logits"] = z.to(_dtype(case["dtype"]))
        z += 0.7 * torch.randn((t, v), generator=g, device=DEV)
        top, idx = torch.topk(z, k, dim=1)
        del z
        st["teacher"], st["idx"] = top.contiguous(), idx.to(torch.int32)
        st["temperature"], st["soft"], st["hard"] = 2.0, 3.0 if case["hard"] else 4.0, 0.25 if case["hard"] else 0.0
        st["targets"] = idx[:, 0].to(torch.int32).contiguous() if case["hard"] else None
        st["row_weight"] = (torch.rand(t, generator=g, device=DEV) > 0.05).float() if t > 8 else None  # 0: padding
        st["scale"] = 1.0 / t
        st["loss"] = torch.empty(t, device=DEV)
        st["grad"] = torch.empty((t, v), dtype=_dtype(case["grad"]), device=DEV) if case["grad"] else None
    return st


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "quant":
        x, _, s = _plain_quant(st["x"])
        return {"x": x.to(torch.bfloat16), "scales": _tiled(s, x.shape[1])}
    if op == "matmul":
        k = st["case"]["k"]
        x, w = _plain_values(st["x"], st["xs"], k), _plain_values(st["w"], st["ws"], k)
        return {"y": (x @ w.t()).to(st["out"].dtype)}
    return _plain_sample(st) if op == "sample" else _plain_distill(st)


def _plain_sample(st):
    """In 64 bits: the sums are long, and a border decides which word is drawn."""
    z = st["logits"].double()
    t, v = z.shape
    greedy = st["temperature"] <= 0
    temp = torch.where(greedy, torch.ones_like(st["temperature"]), st["temperature"]).double()[:, None]
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    w = torch.exp((z - z[:, :1]) / temp)  # the likeliest has 1
    rank = torch.arange(v, device=z.device)
    keep = ~(greedy[:, None] & (rank > 0))
    if st["top_k"] is not None:
        k = torch.where(st["top_k"] <= 0, v, st["top_k"])[:, None]
        keep &= rank < k
    w *= keep
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        cum = torch.cumsum(w, 1)
        w *= (p >= 1) | (rank == 0) | (cum - w < p * cum[:, -1:])
    if st["min_p"] is not None:
        w *= w >= st["min_p"].double()[:, None]
    by_word = torch.zeros_like(w).scatter_(1, order, w)
    cum = torch.cumsum(by_word, 1)
    at = (cum > st["u"].double()[:, None] * cum[:, -1:]).to(torch.uint8).argmax(1)
    return {"tokens": at.to(torch.int32)}


def _plain_distill(st):
    z = st["logits"].float()
    idx, temp, soft, hard = st["idx"].long(), st["temperature"], st["soft"], st["hard"]
    logp = torch.log_softmax(z / temp, dim=1)
    logq = torch.log_softmax(st["teacher"].float() / temp, dim=1)
    q = logq.exp()
    loss = soft * (q * (logq - logp.gather(1, idx))).sum(1)
    d = None
    if st["grad"] is not None:
        d = logp.exp_().scatter_add_(1, idx, -q).mul_(soft / temp)
    if st["targets"] is not None:
        y = st["targets"].long()[:, None]
        logp = torch.log_softmax(z, dim=1)
        loss = loss - hard * logp.gather(1, y)[:, 0]
        if d is not None:
            d += logp.exp_().scatter_add_(1, y, -torch.ones_like(y, dtype=torch.float32)).mul_(hard)
    if st["row_weight"] is not None:
        loss = loss * st["row_weight"]
        if d is not None:
            d *= st["row_weight"][:, None]
    if d is None:
        return {"loss": loss}
    return {"loss": loss, "grad": (d * st["scale"]).to(st["grad"].dtype)}


def _run_own(st):
    import sketch_compressed_sparse_gb300 as s2

    op = st["op"]
    if op == "quant":
        s2.s2_pack4(st["x"], st["codes"], st["scales"])
        s2.s2_unpack4(st["codes"], st["scales"], st["out"])
        return {"x": st["out"], "scales": st["scales"]}
    if op == "matmul":
        s2.s2_matmul4(st["x"], st["xs"], st["w"], st["ws"], st["out"])
        return {"y": st["out"]}
    if op == "sample":
        s2.s2_sample(st["logits"], st["u"], st["tokens"], temperature=st["temperature"], top_k=st["top_k"],
                     top_p=st["top_p"], min_p=st["min_p"])
        return {"tokens": st["tokens"]}
    s2.s2_distill(st["logits"], st["idx"], st["teacher"], st["loss"], st["grad"], targets=st["targets"],
                  row_weight=st["row_weight"], temperature=st["temperature"], soft=st["soft"], hard=st["hard"],
                  scale=st["scale"])
    return {"loss": st["loss"]} if st["grad"] is None else {"loss": st["loss"], "grad": st["grad"]}


def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "quant":
        rows, cols = case["rows"], case["cols"]
        # the input once, the codes, scales and read-back values once
        return {"bytes": rows * (cols * (size + 2) + _up(cols, 2) + _up(cols, B)), "flops": 3 * rows * cols}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (_up(k, 2) + _up(k, B)) + m * n * size, "flops": 2 * m * n * k}
    t, v = case["t"], case["v"]
    if case["op"] == "sample":
        return {"bytes": t * v * size + 24 * t, "flops": 4 * t * v}
    out = {"f32": 4, "bf16": 2, "": 0}[case["grad"]]
    passes = 2 if case["hard"] else 1
    return {"bytes": t * v * (size + out) + 8 * t * case["k"] + 12 * t, "flops": t * v * passes * (5 if out else 3)}


# ---- the definitions in 64 bits, written apart from the above ----

def _exact_quant(x):
    """float64 values (host array) and scale bytes [rows, blocks]."""
    rows, cols = x.shape
    amax = np.maximum.reduceat(np.abs(x), np.arange(_up(cols, B)) * B, axis=1)
    e = np.full(amax.shape, -125.0)
    some = amax > 0
    e[some] = np.ceil(np.log2(amax[some] / 6.0))
    e = np.where(amax > 6.0 * np.exp2(e), e + 1, e)
    e = np.where(some & (amax <= 6.0 * np.exp2(e - 1)), e - 1, e)
    e = np.maximum(e, -125.0)
    s = np.exp2(np.repeat(e, B, axis=1)[:, :cols])
    v = x / s
    step = np.where(np.abs(v) < 2, 0.5, np.where(np.abs(v) < 4, 1.0, 2.0))
    return np.rint(v / step) * step * s, (e + 127).astype(np.uint8)


def _exact_tiles(s, rows, cols):
    out = np.full(_up(rows, 128) * _up(cols, 128) * 512, 127, np.uint8)
    r, j = np.arange(rows)[:, None], np.arange(s.shape[1])[None, :]
    out[(r // 128 * _up(cols, 128) + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4] = s
    return out


def _values64(codes, scales, cols):
    """float64 values of a packed matrix, from its bytes one half at a time."""
    rows = codes.shape[0]
    table = torch.tensor([(-1.0) ** (c >> 3) * (c % 8 * 0.5 if c % 8 < 4 else (2 + c % 2) * 2.0 ** (c % 8 // 2 - 2)) for c in range(16)],
                         dtype=torch.float64, device=DEV)
    v = torch.empty((rows, cols), dtype=torch.float64, device=DEV)
    v[:, 0::2] = table[(codes & 15).long()]
    v[:, 1::2] = table[(codes >> 4).long()[:, :cols // 2]]
    r = torch.arange(rows, device=DEV)
    for j in range(_up(cols, B)):
        at = (r // 128 * _up(cols, 128) + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4
        v[:, j * B:(j + 1) * B] *= torch.exp2(scales[at].double() - 127)[:, None]
    return v


def _exact_tokens(st):
    """Row by row: the kept words one after the other, each filter from its definition."""
    z, got = st["logits"].double(), []
    for i in range(z.shape[0]):
        row, temp = z[i], float(st["temperature"][i])
        if temp <= 0:
            got.append(int(torch.nonzero(row == row.max())[0]))
            continue
        w = torch.exp(row / temp - row.max() / temp)
        rank = torch.empty_like(row, dtype=torch.int64)
        by = torch.argsort(-row, stable=True)
        rank[by] = torch.arange(row.numel(), device=DEV)
        if st["top_k"] is not None and int(st["top_k"][i]) > 0:
            w[rank >= int(st["top_k"][i])] = 0
        if st["top_p"] is not None and float(st["top_p"][i]) < 1:
            mass = torch.cumsum(w[by], 0)
            reached = torch.nonzero(mass >= float(st["top_p"][i]) * w.sum())
            last = int(reached[0]) if len(reached) else row.numel()
            w[rank > last] = 0
        if st["min_p"] is not None:
            w[w < float(st["min_p"][i]) * w.max()] = 0
        mass = torch.cumsum(w, 0)
        got.append(int(torch.nonzero(mass > float(st["u"][i]) * mass[-1])[0]))
    return torch.tensor(got, dtype=torch.int32, device=DEV)


def _exact_distill(st):
    t, v = st["logits"].shape
    temp, soft, hard = st["temperature"], st["soft"], st["hard"]
    loss = torch.empty(t, dtype=torch.float64, device=DEV)
    grad = torch.empty((t, v), dtype=torch.float64, device=DEV) if st["grad"] is not None else None
    for a in range(0, t, 128):
        rows = slice(a, min(t, a + 128))
        z, idx = st["logits"][rows].double(), st["idx"][rows].long()
        at = torch.arange(z.shape[0], device=DEV)
        weight = st["row_weight"][rows].double() if st["row_weight"] is not None else torch.ones(z.shape[0], dtype=torch.float64, device=DEV)
        q = torch.exp(st["teacher"][rows].double() / temp - (st["teacher"][rows].double() / temp).logsumexp(1, keepdim=True))
        lse = (z / temp).logsumexp(1)
        term = torch.where(q > 0, q * (torch.log(q) - z[at[:, None], idx] / temp + lse[:, None]), torch.zeros_like(q))
        one = soft * term.sum(1)
        d = torch.exp(z / temp - lse[:, None]) * (soft / temp)
        for k in range(idx.shape[1]):
            d[at, idx[:, k]] -= q[:, k] * (soft / temp)
        if st["targets"] is not None:
            y = st["targets"][rows].long()
            lse = z.logsumexp(1)
            one = one + hard * (lse - z[at, y])
            d += hard * torch.exp(z - lse[:, None])
            d[at, y] -= hard
        loss[rows] = one * weight
        if grad is not None:
            grad[rows] = d * (weight * st["scale"])[:, None]
    return {"loss": loss} if grad is None else {"loss": loss, "grad": grad}


def exact(case, seed):
    if case["op"] == "quant" and case["rows"] * case["cols"] > 40_000_000:
        return None
    st = prepare(case, seed)
    if case["op"] == "quant":
        x, s = _exact_quant(st["x"].double().cpu().numpy())
        return {"x": x, "scales": _exact_tiles(s, case["rows"], case["cols"])}
    if case["op"] == "matmul":
        k = case["k"]
        return {"y": torch.matmul(_values64(st["x"], st["xs"], k), _values64(st["w"], st["ws"], k).T)}
    return {"tokens": _exact_tokens(st)} if case["op"] == "sample" else _exact_distill(st)
