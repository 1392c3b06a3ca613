"""Cases that measure the 8-bit layer operators: packing to 8 bits with block
scales, unpacking, the product of two packed matrices, and the weight gradient
from a packed activation.

Format: e4m3 codes and one power-of-two scale (a byte b stands for 2^(b-127))
for each block of 128 elements of a row ("rows") or of 128 x 128 elements
("tiles"). With own = False the operators run in plain torch operations in
float32; with own = True through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
B = 128

# The framework's own layers: the large language model's softmax layer
# (267,735 x 1024) and the embedding workload's (33,278 x 512).
LM_ROWS, LM_COLS = 267735, 1024
EMB_ROWS, EMB_COLS = 33278, 512


def listed():
    return [
        # one token's hidden state packed before a serving product: latency
        {"name": "pack_token", "op": "pack", "rows": 1, "cols": LM_COLS, "dtype": "bf16", "tiles": False},
        # a training batch's activations, kept in 8 bits for the backward pass
        {"name": "pack_activations", "op": "pack", "rows": 8192, "cols": 4096, "dtype": "bf16", "tiles": False},
        # a float32 weight after its update: 128 x 128 tiles, both orders
        {"name": "pack_weight", "op": "pack", "rows": EMB_ROWS, "cols": EMB_COLS, "dtype": "f32", "tiles": True},
        # a small ragged checkpoint read back in float32
        {"name": "unpack_ragged", "op": "unpack", "rows": 1999, "cols": 650, "dtype": "f32", "tiles": False},
        # a batch's checkpoint read back in bfloat16
        {"name": "unpack_activations", "op": "unpack", "rows": 8192, "cols": 4096, "dtype": "bf16", "tiles": False},
        # one token through a square layer: latency, and reading the weight
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16"},
        # a few sequences' next-token logits over the large vocabulary, in float32
        {"name": "matmul_serving_head", "op": "matmul", "m": 24, "n": LM_ROWS, "k": LM_COLS, "dtype": "f32"},
        # a hidden layer of a training step
        {"name": "matmul_layer", "op": "matmul", "m": 8192, "n": 4096, "k": 4096, "dtype": "bf16"},
        # a training step's logits over the large vocabulary (odd row length)
        {"name": "matmul_train_head", "op": "matmul", "m": 2048, "n": LM_ROWS, "k": LM_COLS, "dtype": "bf16"},
        # the weight gradient of a small layer from a short batch
        {"name": "wgrad_small", "op": "wgrad", "t": 200, "n": 512, "k": 512, "dtype": "f32"},
        # the weight gradient of a hidden layer
        {"name": "wgrad_layer", "op": "wgrad", "t": 8192, "n": 4096, "k": 4096, "dtype": "bf16"},
        # the large vocabulary's weight gradient, the array that encode reads
        {"name": "wgrad_train_head", "op": "wgrad", "t": 2048, "n": LM_ROWS, "k": LM_COLS, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pack", "unpack", "matmul", "matmul", "wgrad", "wgrad"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("pack", "unpack"):
        rows = _log(rng, 1, 16384)
        cols = _log(rng, 32, 8192)
        while rows * cols > 8192 * 4096:
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "tiles": rng.random() < 0.4}
    most = 2048 * LM_ROWS * LM_COLS // 2
    first, n, k = _log(rng, 1, 8192), _log(rng, 64, LM_ROWS), _log(rng, 64, 4096)
    if rng.random() < 0.5:  # half of the widths are multiples of 8, as layers mostly have
        n, k = -(-n // 8) * 8, -(-k // 8) * 8
    while first * n * k > most or first * n > 1 << 29 or n * k > 1 << 29:
        n = max(64, n // 2)
    return {"op": op, ("m" if op == "matmul" else "t"): first, "n": n, "k": k, "dtype": dtype}


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _blocks(x):
    return -(-x // B)


def _room(rows, cols):
    """An uninitialised code matrix [rows, cols] whose rows start on 16 bytes."""
    return torch.empty((rows, -(-cols // 16) * 16), dtype=torch.uint8, device=DEV)[:, :cols]


def _pow2(b):
    """2^(b-127) of each byte, from the bits of a float32 (1 <= b <= 254)."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _plain_pack(x, tiles):
    """Codes (e4m3 tensor) and scale bytes of x, all finite."""
    rows, cols = x.shape
    nb, rb = _blocks(cols), _blocks(rows)
    v = x.float()
    p = torch.nn.functional.pad(v, (0, nb * B - cols, 0, rb * B - rows if tiles else 0))
    v = p.reshape(rb, B, nb, B) if tiles else p.reshape(rows, 1, nb, B)
    m, ex = torch.frexp(v.abs().amax(dim=(1, 3), keepdim=True))
    # the least e with amax <= 448 * 2^e = 0.875 * 2^(9+e), not below -117
    e = torch.where(m == 0, torch.full_like(ex, -117), (ex - 9 + (m > 0.875)).clamp(min=-117))
    q = (v * _pow2(127 - e)).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(-1, nb * B)[:rows, :cols]
    return q.contiguous().view(torch.float8_e4m3fn), (e + 127).to(torch.uint8).reshape(-1, nb)


def _plain_values(codes, scales, tiles):
    """The float32 values of a packed matrix."""
    rows, cols = codes.shape
    s = _pow2(scales)
    if tiles:
        s = s.repeat_interleave(B, 0)[:rows]
    return codes.view(torch.float8_e4m3fn).float() * s.repeat_interleave(B, 1)[:, :cols]


def _activations(g, rows, cols):
    """Hidden states: unit normal, a few channels and tokens far larger, some tokens zero (padding)."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((1, cols), generator=g, device=DEV))
    x *= 1 + 30 * (torch.rand((1, cols), generator=g, device=DEV) < 0.005)
    if rows > 8:
        x *= torch.rand((rows, 1), generator=g, device=DEV) > 0.02
    return x


def _packed(x, tiles):
    """x as a user holds it packed: codes with rows on 16 bytes, and scale bytes."""
    codes, scales = _plain_pack(x, tiles)
    room = _room(*x.shape)
    room.copy_(codes.view(torch.uint8))
    return room, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"case": case, "op": case["op"], "dtype": _dtype(case)}
    if case["op"] in ("pack", "unpack"):
        rows, cols, tiles = case["rows"], case["cols"], case["tiles"]
        x = torch.randn((rows, cols), generator=g, device=DEV) * cols ** -0.5 if tiles else _activations(g, rows, cols)
        st["tiles"] = tiles
        if case["op"] == "pack":
            st["x"] = x.to(st["dtype"])
            st["codes"] = _room(rows, cols)
            st["scales"] = torch.empty((_blocks(rows) if tiles else rows, _blocks(cols)), dtype=torch.uint8, device=DEV)
            if tiles:
                st["codes_t"] = _room(cols, rows)
                st["scales_t"] = torch.empty((_blocks(cols), _blocks(rows)), dtype=torch.uint8, device=DEV)
        else:
            st["codes"], st["scales"] = _packed(x, tiles)
            st["out"] = torch.empty((rows, cols), dtype=st["dtype"], device=DEV)
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"], st["xs"] = _packed(_activations(g, m, k), False)
        st["w"], st["ws"] = _packed(torch.randn((n, k), generator=g, device=DEV) * k ** -0.5, True)
        st["out"] = torch.empty((m, n), dtype=st["dtype"], device=DEV)
    else:
        t, n, k = case["t"], case["n"], case["k"]
        st["x"], st["xs"] = _packed(_activations(g, t, k), False)
        # output gradients: heavy-tailed over the row, scaled by the batch
        dy = torch.randn((t, n), generator=g, device=DEV)
        dy = dy * dy.abs().square_() / t
        st["dy"] = dy.to(torch.bfloat16)
        st["out"] = torch.empty((n, k), dtype=st["dtype"], device=DEV)
    return st


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "pack":
        codes, scales = _plain_pack(st["x"], st["tiles"])
        r = {"codes": codes, "scales": scales}
        if st["tiles"]:
            r["codes_t"] = codes.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)
            r["scales_t"] = scales.t().contiguous()
        return r
    if op == "unpack":
        return {"x": _plain_values(st["codes"], st["scales"], st["tiles"]).to(st["dtype"])}
    if op == "matmul":
        x = _plain_values(st["x"], st["xs"], False)
        w = _plain_values(st["w"], st["ws"], True)
        return {"y": (x @ w.t()).to(st["dtype"])}
    x = _plain_values(st["x"], st["xs"], False)
    return {"dw": (st["dy"].float().t() @ x).to(st["dtype"])}


def _run_own(st):
    import sketch_compressed_sparse_gb300 as s2

    op = st["op"]
    if op == "pack":
        f8 = torch.float8_e4m3fn
        if st["tiles"]:
            s2.s2_pack8(st["x"], st["codes"], st["scales"], "tiles", st["codes_t"], st["scales_t"])
            return {"codes": st["codes"].view(f8), "scales": st["scales"],
                    "codes_t": st["codes_t"].view(f8), "scales_t": st["scales_t"]}
        s2.s2_pack8(st["x"], st["codes"], st["scales"])
        return {"codes": st["codes"].view(f8), "scales": st["scales"]}
    if op == "unpack":
        s2.s2_unpack8(st["codes"], st["scales"], st["out"], "tiles" if st["tiles"] else "rows")
        return {"x": st["out"]}
    if op == "matmul":
        s2.s2_matmul8(st["x"], st["xs"], st["w"], st["ws"], st["out"])
        return {"y": st["out"]}
    s2.s2_wgrad8(st["dy"], st["x"], st["xs"], st["out"])
    return {"dw": st["out"]}


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("pack", "unpack"):
        rows, cols, tiles = case["rows"], case["cols"], case["tiles"]
        copies = 2 if tiles and case["op"] == "pack" else 1
        scales = (_blocks(rows) if tiles else rows) * _blocks(cols)
        return {"bytes": rows * cols * (size + copies) + scales * copies, "flops": 2 * rows * cols}
    n, k = case["n"], case["k"]
    first = case["m"] if case["op"] == "matmul" else case["t"]
    flops = 2 * first * n * k
    xbytes = first * k + first * _blocks(k)
    if case["op"] == "matmul":
        return {"bytes": xbytes + n * k + _blocks(n) * _blocks(k) + first * n * size, "flops": flops}
    return {"bytes": xbytes + 2 * first * n + n * k * size, "flops": flops}


# ---- the definitions in 64 bits, written apart from the above ----

def _code_table():
    t = np.empty(256)
    for c in range(256):
        ex, man = (c >> 3) & 15, c & 7
        v = math.nan if (ex, man) == (15, 7) else man * 2.0 ** -9 if ex == 0 else (8 + man) * 2.0 ** (ex - 10)
        t[c] = -v if c & 128 else v
    return t


def _values64(codes, scales, tiles):
    """float64 values of a packed matrix, block column by block column."""
    rows, cols = codes.shape
    out = torch.from_numpy(_code_table()).to(DEV)[codes.to(torch.int32)]
    f = torch.exp2(scales.double() - 127)
    if tiles:
        f = f[torch.arange(rows, device=DEV) // B]
    for j in range(_blocks(cols)):
        out[:, j * B:(j + 1) * B] *= f[:, j:j + 1]
    return out


def _exact_pack(x, tiles):
    """float64 code values and integer scale bytes of a matrix on the host."""
    rows, cols = x.shape
    rb, nb = (_blocks(rows) if tiles else rows), _blocks(cols)
    height = B if tiles else 1
    starts_c = np.arange(nb) * B
    amax = np.maximum.reduceat(np.abs(x), starts_c, axis=1)
    if tiles:
        amax = np.maximum.reduceat(amax, np.arange(rb) * B, axis=0)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(amax / 448.0))
    e = np.where(amax > 0, e, -117.0)
    e = np.where(amax > 448.0 * np.exp2(e), e + 1, e)
    e = np.where((amax > 0) & (amax <= 448.0 * np.exp2(e - 1)), e - 1, e)
    e = np.maximum(e, -117.0)
    s = np.repeat(np.repeat(e, height, axis=0)[:rows], B, axis=1)[:, :cols]
    v = x / np.exp2(s)
    with np.errstate(divide="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(np.abs(v))), -6.0) - 3.0)
    return np.rint(v / step) * step, (e + 127).astype(np.uint8)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "pack":
        codes, scales = _exact_pack(st["x"].double().cpu().numpy(), st["tiles"])
        r = {"codes": codes, "scales": scales}
        if st["tiles"]:
            r["codes_t"], r["scales_t"] = codes.T.copy(), scales.T.copy()
        return r
    if op == "unpack":
        return {"x": _values64(st["codes"], st["scales"], st["tiles"])}
    x = _values64(st["x"], st["xs"], False)
    if op == "matmul":
        w = _values64(st["w"], st["ws"], True)
        return {"y": torch.matmul(x, w.T)}
    return {"dw": torch.matmul(st["dy"].double().T, x)}
