"""Timed cases of the 4-bit merged weight and of dropout from a counter-based generator.

Four operators of the quantised fine-tuning layer, each as a user calls it (``own`` true) and
in a plain form of elementary torch operations (``own`` false):

  merge    the 4-bit merged weight (codes, group scales) from W0 and two index maps, read back
  product  y = x W^T, or dx = dy W, with the 4-bit weight W, from one token to thousands
  layer    the POET-X linear on the 4-bit weight: a forward pass for a few tokens, or a training
           step (forward, dx, dG) with dropout of its input
  dropout  dropout with a mask that is never stored, alone or fused with an index map

4-bit format.  codes: uint8 [n/128, m, 64]; the 64 bytes of a row's 128-column block are four
16-byte chunks t of four little-endian 32-bit words w; nibble p of a word holds q + 8 of column
32 w + 8 t + e with p = e // 2 + 4 (e % 2).  scales: bf16 [n/128, m, 128/group].
Scale of a group: max|w| / 7 rounded to 5 significant bits (nearest even), so that s q is a bf16
number; q = nearest integer to w / s (ties to even), in [-7, 7].

Dropout mask.  Philox4x32-10 with key = seed and counter = (column // 8, row, site, step); lane
column % 8 takes 16 of the 128 bits (low half of word 0 first) and the value is kept when they
are >= thr = round(65536 p), multiplied by 65536 / (65536 - thr).
"""
import numpy as np
import torch

own = False

DEV = "cuda"
E_ORDER = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble that holds element e of a word


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a square attention projection's weight brought to 4 bits under new permutations
        {"name": "merge bf16 5120x5120 g128", "op": "merge", "m": 5120, "n": 5120, "group": 128,
         "dtype": "bf16", "perm": True},
        # an fp32 checkpoint's up-projection, fine groups
        {"name": "merge f32 13824x5120 g32", "op": "merge", "m": 13824, "n": 5120, "group": 32,
         "dtype": "f32", "perm": True},
        # one new token through an attention projection: the smallest call, latency counts
        {"name": "product T1 5120x5120 g128", "op": "product", "T": 1, "m": 5120, "n": 5120,
         "group": 128, "transpose": False},
        # a handful of sequences' next tokens through the up-projection
        {"name": "product T6 13824x5120 g64", "op": "product", "T": 6, "m": 13824, "n": 5120,
         "group": 64, "transpose": False},
        # a long batch of tokens: the largest work
        {"name": "product T8192 13824x5120 g128", "op": "product", "T": 8192, "m": 13824,
         "n": 5120, "group": 128, "transpose": False},
        # gradient through the frozen down-projection for one token
        {"name": "product^T T1 5120x13824 g32", "op": "product", "T": 1, "m": 5120, "n": 13824,
         "group": 32, "transpose": True},
        # gradient of a short ragged batch, a row count that no tile divides
        {"name": "product^T T53 4999x4096 g64", "op": "product", "T": 53, "m": 4999, "n": 4096,
         "group": 64, "transpose": True},
        # decoding: the whole layer for one token
        {"name": "layer T1 5120x5120 g128", "op": "layer", "T": 1, "m": 5120, "n": 5120, "b": 256,
         "group": 128, "step": False, "p": 0.0},
        # a training step of the up-projection with dropout of its input
        {"name": "layer step T4096 13824x5120 g64", "op": "layer", "T": 4096, "m": 13824,
         "n": 5120, "b": 256, "group": 64, "step": True, "p": 0.1},
        # dropout alone, fp32, odd sizes (unaligned rows)
        {"name": "dropout f32 3001x5003", "op": "dropout", "T": 3001, "n": 5003, "dtype": "f32",
         "p": 0.25, "mode": "plain"},
        # the layer's input: dropout fused with the permutation, forward direction
        {"name": "dropout+perm bf16 8192x5120", "op": "dropout", "T": 8192, "n": 5120,
         "dtype": "bf16", "p": 0.1, "mode": "gather"},
        # its gradient: the inverse permutation, then the same mask (wide rows)
        {"name": "dropout+perm^T bf16 4096x13824", "op": "dropout", "T": 4096, "n": 13824,
         "dtype": "bf16", "p": 0.1, "mode": "scatter"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["merge", "product", "product", "layer", "dropout"])
    group = rng.choice([32, 64, 128])
    if op == "merge":
        return {"op": op, "m": _log(rng, 64, 13824), "n": 128 * _log(rng, 1, 40),
                "group": group, "dtype": rng.choice(["bf16", "f32"]),
                "perm": rng.random() < 0.8}
    if op == "product":
        T = _log(rng, 1, 8192)
        # whole tiles for long batches, any row count for short ones
        m = 256 * _log(rng, 2, 54) if T > 64 else _log(rng, 256, 13824)
        return {"op": op, "T": T, "m": m, "n": 256 * _log(rng, 2, 20), "group": group,
                "transpose": rng.random() < 0.5}
    if op == "layer":
        b = rng.choice([128, 256, 512])
        step = rng.random() < 0.5
        return {"op": op, "T": _log(rng, 200, 4096) if step else _log(rng, 1, 64),
                "m": b * _log(rng, 1, 6656 // b), "n": b * _log(rng, 1, 5120 // b), "b": b,
                "group": group, "step": step, "p": rng.choice([0.05, 0.1, 0.3]) if step else 0.0}
    mode = rng.choice(["plain", "gather", "scatter"])
    dtype = rng.choice(["bf16", "f32"])
    return {"op": op, "T": _log(rng, 1, 8192), "n": _log(rng, 64, 6000), "dtype": dtype,
            "p": rng.choice([0.05, 0.1, 0.25, 0.5]), "mode": mode}


def work(c):
    if c["op"] == "merge":
        mn = c["m"] * c["n"]
        es = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": mn * es + mn / 2 + 2 * mn / c["group"] + 2 * mn, "flops": 2 * mn}
    if c["op"] == "product":
        mn = c["m"] * c["n"]
        return {"bytes": mn / 2 + 2 * mn / c["group"] + 2 * c["T"] * (c["m"] + c["n"]),
                "flops": 2 * c["T"] * mn}
    if c["op"] == "layer":
        T, m, n, b = c["T"], c["m"], c["n"], c["b"]
        byts = m * n / 2 + 2 * m * n / c["group"] + 2 * (m + n) * b + 2 * T * (m + n) + 4 * (m + n)
        flops = 2 * T * (m * n + (m + n) * b)
        if c["step"]:  # also x, dy in and dx out, the index maps' inverses, dG out
            byts += 2 * T * (m + n) + 4 * (m + n) * b + 4 * (m + n)
            flops += 2 * T * (m * n + 2 * (m + n) * b)
        return {"bytes": byts, "flops": flops}
    es = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": 2 * es * c["T"] * c["n"], "flops": c["T"] * c["n"]}


# ------------------------------------------------------------------------------- inputs
def _quantise(W, group):
    """q (integers as float32) [m, n] and s (float32) [m, n / group] of W (float32)."""
    m, n = W.shape
    Wg = W.view(m, n // group, group)
    bits = (Wg.abs().amax(2) / 7).view(torch.int32)
    bits = (bits + 0x3FFFF + ((bits >> 19) & 1)) & -0x80000  # 5 significant bits, nearest even
    s = bits.view(torch.float32)
    safe = torch.where(s > 0, s, torch.ones_like(s))
    q = torch.round(Wg.double() / safe.double().unsqueeze(2)).clamp_(-7, 7).float()
    return q.view(m, n), s


def _pack(q):
    m, n = q.shape
    u = (q + 8).to(torch.uint8).view(m, n // 128, 4, 4, 8).permute(1, 0, 3, 2, 4)  # [nb,m,t,w,e]
    nib = torch.empty_like(u, memory_format=torch.contiguous_format)
    nib[..., E_ORDER] = u
    nib = nib.view(n // 128, m, 64, 2)
    return (nib[..., 0] | (nib[..., 1] << 4)).contiguous()


def _pack_scales(s, group):
    m = s.shape[0]
    return s.view(m, -1, 128 // group).permute(1, 0, 2).to(torch.bfloat16).contiguous()


def _unpack(codes, scales, group):
    """The weight [m, n] in float32 that codes and scales stand for."""
    nb, m, _ = codes.shape
    nib = torch.stack((codes & 15, codes >> 4), 3).view(nb, m, 4, 4, 8)[..., E_ORDER]  # [..t,w,e]
    q = nib.permute(1, 0, 3, 2, 4).reshape(m, nb * 128).float() - 8
    s = scales.float().permute(1, 0, 2).reshape(m, -1)
    return (q.view(m, -1, group) * s.unsqueeze(2)).view(m, nb * 128)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    def perm(k):
        p = torch.randperm(k, generator=g, device=DEV)
        return p.to(torch.int32), torch.argsort(p).to(torch.int32)

    st = {"c": c, "seed": int(seed)}
    bf = torch.bfloat16
    if c["op"] == "merge":
        dt = bf if c["dtype"] == "bf16" else torch.float32
        st["W"] = normal(c["m"], c["n"], dtype=dt, scale=c["n"] ** -0.5)
        st["pR"], st["pP"] = (perm(c["m"])[0], perm(c["n"])[0]) if c["perm"] else (None, None)
        st["q"] = torch.empty(c["n"] // 128, c["m"], 64, dtype=torch.uint8, device=DEV)
        st["s"] = torch.empty(c["n"] // 128, c["m"], 128 // c["group"], dtype=bf, device=DEV)
        st["out"] = torch.empty(c["m"], c["n"], dtype=bf, device=DEV)
    elif c["op"] in ("product", "layer"):
        T, m, n = c["T"], c["m"], c["n"]
        q, s = _quantise(normal(m, n, dtype=torch.float32, scale=n ** -0.5), c["group"])
        st["q"], st["s"] = _pack(q), _pack_scales(s, c["group"])
        del q, s
        if c["op"] == "product":
            st["x"] = normal(T, m if c["transpose"] else n)
            st["y"] = torch.empty(T, n if c["transpose"] else m, dtype=bf, device=DEV)
        else:
            b = c["b"]
            for side, k in (("P", n), ("R", m)):
                st["p" + side], st["i" + side] = perm(k)
                Q = normal(k // b, b, b, dtype=torch.float32, scale=0.01)
                Q = torch.triu(Q, 1)
                Q = Q - Q.transpose(1, 2)
                eye = torch.eye(b, device=DEV)
                st["G" + side] = (eye + 2 * Q + 2 * torch.bmm(Q, Q)).to(bf)
            st["x"], st["y"] = normal(T, n), torch.empty(T, m, dtype=bf, device=DEV)
            st["step"] = torch.full((1,), 17, dtype=torch.int64, device=DEV)
            if c["step"]:
                st["dy"], st["dx"] = normal(T, m), torch.empty(T, n, dtype=bf, device=DEV)
                st["U"], st["W"] = torch.empty_like(st["dx"]), torch.empty_like(st["y"])
                st["dGP"] = torch.empty(n // b, b, b, device=DEV)
                st["dGR"] = torch.empty(m // b, b, b, device=DEV)
    else:
        dt = bf if c["dtype"] == "bf16" else torch.float32
        st["x"] = normal(c["T"], c["n"], dtype=dt)
        st["out"] = torch.empty_like(st["x"])
        st["idx"] = perm(c["n"])[0]
        st["step"] = torch.full((1,), 17, dtype=torch.int64, device=DEV)
    return st


# ------------------------------------------------------------------------------- plain forms
def _mulhilo(a, b):
    """High and low 32 bits of a * b for a an int64 tensor below 2**32 and b an int."""
    lo_part = a * (b & 0xFFFF)
    hi_part = a * (b >> 16) + (lo_part >> 16)
    return hi_part >> 16, ((hi_part & 0xFFFF) << 16) | (lo_part & 0xFFFF)


def _philox(c0, c1, c2, c3, k0, k1):
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c0, c1, c2, c3


def _factor(T, n, p, seed, step):
    """What dropout multiplies by [T, n], float32: 0 or 65536 / (65536 - thr)."""
    thr = int(p * 65536 + 0.5)
    calls = (n + 7) // 8
    zero = torch.zeros(T, calls, dtype=torch.int64, device=DEV)
    c0 = zero + torch.arange(calls, device=DEV)
    c1 = zero + torch.arange(T, device=DEV).view(T, 1)
    words = _philox(c0, c1, zero + SITE, zero + step, seed & 0xFFFFFFFF, seed >> 32)
    half = torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], 2).view(T, calls * 8)
    return (half[:, :n] >= thr).float() * (65536.0 / (65536 - thr))


SITE = 3


def _blocks(x, G, b):
    """x's b-wide column blocks times G_j^T."""
    T = x.shape[0]
    return torch.bmm(x.view(T, -1, b).transpose(0, 1), G.transpose(1, 2)).transpose(0, 1).reshape(
        T, -1)


def _block_grads(a, x, b):
    T = a.shape[0]
    return torch.bmm(a.view(T, -1, b).permute(1, 2, 0), x.view(T, -1, b).transpose(0, 1))


def _plain(st):
    c = st["c"]
    bf = torch.bfloat16
    if c["op"] == "merge":
        W = st["W"].float()
        if c["perm"]:
            W = W[st["pR"].long()][:, st["pP"].long()].contiguous()
        q, s = _quantise(W, c["group"])
        return {"w": (q.view(c["m"], -1, c["group"]) * s.unsqueeze(2)).view_as(q).to(bf),
                "s": _pack_scales(s, c["group"])}
    if c["op"] == "product":
        W = _unpack(st["q"], st["s"], c["group"])
        x = st["x"].float()
        return torch.matmul(x, W if c["transpose"] else W.t()).to(bf)
    if c["op"] == "layer":
        b, m, n = c["b"], c["m"], c["n"]
        W0 = _unpack(st["q"], st["s"], c["group"])
        GP, GR = st["GP"].float(), st["GR"].float()
        x = st["x"].float()
        if c["step"]:
            factor = _factor(c["T"], n, c["p"], st["seed"], 17)
            x = x * factor
        U = x[:, st["pP"].long()]
        W = torch.matmul(_blocks(U, GP, b), W0.t())
        y = _blocks(W, GR, b)[:, st["iR"].long()].to(bf)
        if not c["step"]:
            return y
        dZ = st["dy"].float()[:, st["pR"].long()]
        dGR = _block_grads(dZ, W, b)
        dV = torch.matmul(_blocks(dZ, GR.transpose(1, 2), b), W0)
        dGP = _block_grads(dV, U, b)
        dx = (_blocks(dV, GP.transpose(1, 2), b)[:, st["iP"].long()] * factor).to(bf)
        return {"y": y, "dx": dx, "dGP": dGP.to(bf), "dGR": dGR.to(bf)}
    factor = _factor(c["T"], c["n"], c["p"], st["seed"], 17)
    x, idx = st["x"].float(), st["idx"].long()
    if c["mode"] == "gather":
        out = (x * factor)[:, idx]
    elif c["mode"] == "scatter":
        out = x[:, idx] * factor
    else:
        out = x * factor
    return out.to(st["x"].dtype)


# ------------------------------------------------------------------------------- the framework
def _own(st):
    from orthogonal_reparameterized_cnp_b200 import poetx as P
    c = st["c"]
    if c["op"] == "merge":
        P.merge_perm_q4(st["W"], st["q"], st["s"], st["pR"], st["pP"], c["group"])
        P.dequantize_q4(st["q"], st["s"], st["out"], c["group"])
        return {"w": st["out"], "s": st["s"]}
    if c["op"] == "product":
        P.matmul_q4(st["x"], st["q"], st["s"], st["y"], c["group"], transpose=c["transpose"])
        return st["y"]
    if c["op"] == "dropout":
        drop = P.dropout_desc(c["p"], st["seed"], site=SITE, step=st["step"])
        if c["mode"] == "plain":
            P.dropout(drop, st["x"], st["out"])
        else:
            P.permute_cols_dropout(drop, st["x"], st["out"], st["idx"],
                                   mask_output=c["mode"] == "scatter")
        return st["out"]
    weight = P.linear_weight_q4(st["q"], st["s"], c["group"])
    desc = P.linear_desc(c["T"], c["n"], c["m"], c["b"], P.POETX_BF16, st["pP"], st["iP"],
                         st["pR"], st["iR"])
    drop = P.dropout_desc(c["p"], st["seed"], site=SITE, step=st["step"]) if c["step"] else None
    if "ws" not in st:  # kept by the program, as the layer objects keep theirs
        st["ws"] = torch.empty(max(P.linear_ex_workspace(desc, weight, c["step"], c["step"]), 16),
                               dtype=torch.uint8, device=DEV)
    if not c["step"]:
        P.linear_fwd_ex(desc, weight, drop, st["x"], st["GP"], st["GR"], st["y"], None, None,
                        st["ws"])
        return st["y"]
    P.linear_fwd_ex(desc, weight, drop, st["x"], st["GP"], st["GR"], st["y"], st["U"], st["W"],
                    st["ws"])
    P.linear_bwd_ex(desc, weight, drop, st["x"], st["dy"], st["GP"], st["GR"], st["U"], st["W"],
                    st["dx"], st["dGP"], st["dGR"], 0, st["ws"])
    # the gradients of G at the precision of the stored activations that make them
    return {"y": st["y"], "dx": st["dx"], "dGP": st["dGP"].to(torch.bfloat16),
            "dGR": st["dGR"].to(torch.bfloat16)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------- 64 bits
def _exact_weight(st, group):
    """The weight in float64, bit by bit from the packed words."""
    nb, m, _ = st["q"].shape
    words = st["q"].view(torch.int32).to(torch.int64) & 0xFFFFFFFF  # [nb, m, 16 = 4 t + w]
    W = torch.empty(m, nb * 128, dtype=torch.float64, device=DEV)
    for t in range(4):
        for w in range(4):
            for e in range(8):
                col = 32 * w + 8 * t + e
                u = (words[:, :, 4 * t + w] >> (4 * (e // 2 + 4 * (e % 2)))) & 15
                s = st["s"][:, :, col // group].double()
                W[:, col::128] = ((u - 8) * s).t()
    return W


def _exact_factor(T, n, p, seed, step):
    """Dropout's factors in float64, from Philox in numpy's 64-bit unsigned integers."""
    m32 = np.uint64(0xFFFFFFFF)
    calls = -(-n // 8)
    ctr = [np.tile(np.arange(calls, dtype=np.uint64), T),
           np.repeat(np.arange(T, dtype=np.uint64), calls),
           np.full(T * calls, SITE, np.uint64), np.full(T * calls, step, np.uint64)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(b >> np.uint64(32)) ^ ctr[1] ^ np.uint64(key[0]), b & m32,
               (a >> np.uint64(32)) ^ ctr[3] ^ np.uint64(key[1]), a & m32]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    raw = np.stack(ctr, 1).astype("<u4").view("<u2").reshape(T, calls * 8)[:, :n]
    thr = int(np.floor(p * 65536 + 0.5))
    f = np.where(raw >= thr, 65536.0 / (65536 - thr), 0.0)
    return torch.from_numpy(f).to(DEV)


def _dense(G, p):
    """Pi^T blockdiag(G) Pi in float64, with (Pi x)_i = x[p[i]]."""
    D = torch.block_diag(*G.double())
    out = torch.zeros_like(D)
    p = p.long()
    out[p.unsqueeze(1), p.unsqueeze(0)] = D
    return out


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "merge":
        W = st["W"].double()
        if c["perm"]:
            W = W.index_select(0, st["pR"].long()).index_select(1, st["pP"].long())
        W = W.reshape(c["m"], -1, c["group"])
        a = W.abs().max(dim=2).values / 7
        mant, exp = torch.frexp(a)  # a = mant 2^exp, mant in [1/2, 1): 5 bits of it
        s = torch.ldexp(torch.round(mant * 32) / 32, exp)
        q = torch.where(s.unsqueeze(2) > 0, torch.round(W / s.unsqueeze(2)), torch.zeros_like(W))
        w = torch.clamp(q, -7, 7) * s.unsqueeze(2)
        return {"w": w.reshape(c["m"], -1),
                "s": s.reshape(c["m"], -1, 128 // c["group"]).permute(1, 0, 2)}
    if c["op"] == "product":
        W = _exact_weight(st, c["group"])
        return st["x"].double() @ (W if c["transpose"] else W.T)
    if c["op"] == "layer":
        b = c["b"]
        # y = x (R W0 P)^T with the unpermuted weight W0 and the dense rotations R, P
        W0 = _exact_weight(st, c["group"])[st["iR"].long()][:, st["iP"].long()]
        R, Pm = _dense(st["GR"], st["pR"]), _dense(st["GP"], st["pP"])
        x = st["x"].double()
        if c["step"]:
            f = _exact_factor(c["T"], c["n"], c["p"], st["seed"], 17)
            x = x * f
        h = x @ Pm.T @ W0.T
        y = h @ R.T
        if not c["step"]:
            return y
        dy = st["dy"].double()
        dh = dy @ R @ W0
        dx = (dh @ Pm) * f

        def blocks(left, right, p):  # diagonal blocks of (left Pi^T)^T (right Pi^T)
            p = p.long()
            lb, rb = left[:, p], right[:, p]
            return torch.stack([lb[:, j:j + b].T @ rb[:, j:j + b]
                                for j in range(0, lb.shape[1], b)])

        return {"y": y, "dx": dx, "dGP": blocks(dh, x, st["pP"]),
                "dGR": blocks(dy, h, st["pR"])}
    f = _exact_factor(c["T"], c["n"], c["p"], st["seed"], 17)
    x, idx = st["x"].double(), st["idx"].long()
    if c["mode"] == "gather":
        return (x * f).index_select(1, idx)
    if c["mode"] == "scatter":
        return x.index_select(1, idx) * f
    return x * f
