"""Cases of the MoE-block operators: the norm between blocks, the router, the experts and the
4-bit linear, each in a plain form and through the library's entry points.

One MoE block of a decoding step, as the adapters' deltas meet it:

    norm    residual' = residual + s * gate * rms(y; post);  x = rms(residual'; pre)
    route   the topk largest of the router's logits, softmax weights
    moe     out[t] = sum_k w[t,k] * down[e] . (silu(gate[e] . x[t]) * (up[e] . x[t]))
    linear  out[t] = w . x[t], w held in 4 bits with a scale for each group of inputs

4-bit weights. Kp is K rounded up to 256. A row holds Kp / 2 bytes: 32-bit little-endian words,
sixteen to a block of 128 inputs. Word 4 * t + i of a block (t, i < 4) holds the inputs
32 * i + 8 * t + (0 .. 7): input j in bits 4 * (j / 2) where j is even, 16 + 4 * (j / 2) where odd.
The value is scale[row, input / group] * (q - 8). Padding inputs take no part.

`own` false: elementary torch operations in 32 bits. `own` true: the library's calls.
"""

import math

import torch

own = False

EPS = 1e-6
LOWEST = -3.0e38


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decoding step of 23 requests (the repository's decode workload): one small launch
        dict(name="norm-decode", op="norm", T=23, H=2048, post=True, gate="row", strided=False),
        # a prefill chunk, a gate for each token, block output rows inside a wider buffer
        dict(name="norm-prefill", op="norm", T=8192, H=2048, post=True, gate="token", strided=True),
        # 128 experts, top-8, the same decoding step
        dict(name="route-decode", op="route", T=23, E=128, k=8, dtype="f32", renorm=True,
             masked=0.0),
        # an expert-parallel prefill: 256 experts, some masked by the placement
        dict(name="route-prefill", op="route", T=8192, E=256, k=8, dtype="bf16", renorm=False,
             masked=0.1),
        # one request alone: eight experts' weights and no more
        dict(name="moe-one-token", op="moe", fmt="bf16", G=0, T=1, E=128, k=8, H=2048, I=768,
             drop=0.0, hot=0, delta=False),
        # the decode workload's base experts
        dict(name="moe-decode", op="moe", fmt="bf16", G=0, T=23, E=128, k=8, H=2048, I=768,
             drop=0.0, hot=0, delta=False),
        # verify tokens over few experts, odd sizes, a quarter of the pairs on other devices, one
        # expert that every token takes, adapters' deltas added on both products
        dict(name="moe-ragged-adapters", op="moe", fmt="bf16", G=0, T=61, E=40, k=6, H=1032, I=712,
             drop=0.25, hot=1, delta=True),
        # one request, 4-bit experts
        dict(name="moe-w4-one-token", op="moe", fmt="w4", G=128, T=1, E=128, k=8, H=2048, I=768,
             drop=0.0, hot=0, delta=False),
        # sixteen requests with six verify tokens each, 4-bit experts with fine groups
        dict(name="moe-w4-verify", op="moe", fmt="w4", G=32, T=96, E=128, k=8, H=2048, I=768,
             drop=0.0, hot=0, delta=False),
        # an attention projection of one token: a few microseconds of weights
        dict(name="linear-one-token", op="linear", T=1, K=2048, N=2560, G=128),
        # the same kind of projection for a batch, an odd number of outputs
        dict(name="linear-batch", op="linear", T=16, K=4096, N=6151, G=64),
        # an output head over a large vocabulary
        dict(name="linear-head", op="linear", T=5, K=2048, N=120001, G=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _expert_bytes(c):
    n = 3 * c["H"] * c["I"]
    return n * 2.0 if c["fmt"] == "bf16" else n * (0.5 + 2.0 / c["G"])


def draw(rng):
    op = rng.choice(["norm", "route", "moe", "moe", "moe", "linear"])
    while True:
        if op == "norm":
            c = dict(op=op, T=_log(rng, 1, 8192), H=8 * _log(rng, 16, 1024),
                     post=rng.random() < 0.7, gate=rng.choice(["none", "row", "token"]),
                     strided=rng.random() < 0.4)
            sizes, ok = (c["H"],), c["T"] * c["H"] <= 8192 * 2048
        elif op == "route":
            c = dict(op=op, T=_log(rng, 1, 8192), E=_log(rng, 4, 512), k=rng.randint(1, 10),
                     dtype=rng.choice(["f32", "bf16"]), renorm=rng.random() < 0.5,
                     masked=rng.choice([0.0, 0.1, 0.6]))
            sizes = (c["E"],)
            ok = (c["k"] <= c["E"] and c["T"] * c["E"] <= 8192 * 256
                  and not (c["renorm"] and c["k"] == 1))
        elif op == "moe":
            fmt = rng.choice(["bf16", "w4"])
            c = dict(op=op, fmt=fmt, G=rng.choice([32, 64, 128]) if fmt == "w4" else 0,
                     T=_log(rng, 1, 128), E=_log(rng, 4, 256), k=rng.randint(1, 8),
                     H=8 * _log(rng, 16, 512), I=8 * _log(rng, 8, 256),
                     drop=rng.choice([0.0, 0.0, 0.25, 0.5]), hot=rng.choice([0, 0, 1]),
                     delta=rng.random() < 0.3)
            sizes = (c["H"], c["I"], 2 * c["I"], c["H"] // 2, c["I"] // 2)
            per = c["H"] * c["I"]
            ok = (c["hot"] < c["k"] < c["E"] and (c["drop"] == 0 or c["T"] * c["k"] >= 16)
                  and c["E"] * per <= 128 * 2048 * 768
                  and c["T"] * c["k"] * per <= 96 * 8 * 2048 * 768)
        else:
            c = dict(op=op, T=_log(rng, 1, 32), K=8 * _log(rng, 16, 700), N=_log(rng, 64, 120000),
                     G=rng.choice([32, 64, 128]))
            sizes, ok = (c["K"], c["N"], c["K"] // 2), c["N"] * c["K"] <= 120000 * 2048
        if ok and 3072 not in (c["T"], *sizes):
            return c


# -------------------------------------------------------------------------------------- the inputs
def _pad(K):
    return (K + 255) // 256 * 256


def _w4(g, lead, K, G):
    """4-bit rows of K inputs as they come from rounding a normal weight: bytes and scales."""
    Kp = _pad(K)
    n = math.prod(lead)
    q = torch.empty(n, Kp // 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // Kp)
    for r in range(0, n, step):
        m = min(step, n - r)
        v = torch.randn(m, Kp, generator=g, device="cuda").mul_(2.7).round_().clamp_(-8, 7).add_(8)
        v = v.to(torch.uint8).view(m, Kp // 2, 2)
        q[r:r + m] = v[..., 0] | (v[..., 1] << 4)
    s = torch.rand(n, Kp // G, generator=g, device="cuda").mul_(0.8).add_(0.6)
    s = (s / (2.7 * math.sqrt(K))).to(torch.bfloat16)
    return q.view(*lead, Kp // 2), s.view(*lead, Kp // G)


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)


def _weights(g, lead, K):
    out = torch.empty(*lead, K, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(K ** -0.5)
    return out


def _routing(c, g):
    """ids [T, k]: distinct experts of each token (`hot` of them the same for all), some dropped."""
    score = torch.rand(c["T"], c["E"], generator=g, device="cuda")
    if c["hot"]:
        at = int(torch.randint(c["E"], (1,), generator=g, device="cuda"))
        score[:, at] = 2.0
    ids = score.argsort(1, descending=True)[:, :c["k"]].to(torch.int32)
    gone = torch.rand(ids.shape, generator=g, device="cuda") < c["drop"]
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        wide = H + 64 if c["strided"] else H
        y = _normal(g, (T, wide), 3.0)[:, :H]
        s = dict(c=c, y=y, residual=_normal(g, (T, H), 2.0),
                 post=_normal(g, (H,), 0.2) + 1 if c["post"] else None,
                 pre=_normal(g, (H,), 0.2) + 1, scale=0.75, gate=None)
        if c["gate"] != "none":
            s["gate"] = _normal(g, (T, H) if c["gate"] == "token" else (H,), 0.5)
        y[T // 2] = 0  # a block that wrote nothing for one token
        return s
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        v = torch.randn(T, E, generator=g, device="cuda").mul_(2.0)
        v = v.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        gone = torch.rand(T, E, generator=g, device="cuda") < c["masked"]
        v = v.masked_fill(gone, -math.inf)
        if c["masked"] and T >= 4:
            v[T // 2] = -math.inf   # a token that no expert may take
            v[T // 3, 1:] = LOWEST  # one expert, the others at the type's lowest values
        return dict(c=c, logits=v, k=c["k"], renorm=c["renorm"], scale=1.0 if c["renorm"] else 2.5)
    if c["op"] == "linear":
        q, sc = _w4(g, (c["N"],), c["K"], c["G"])
        return dict(c=c, x=_normal(g, (c["T"], c["K"])), w=(q, sc, c["K"], c["G"]))
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    s = dict(c=c, x=_normal(g, (T, H)), ids=_routing(c, g))
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    s["w"] = (w / w.sum(1, keepdim=True)).contiguous()
    if c["fmt"] == "bf16":
        s["gu"], s["dn"] = _weights(g, (E, 2 * I), H), _weights(g, (E, H), I)
    else:
        s["gu"] = (*_w4(g, (E, 2 * I), H, c["G"]), H, c["G"])
        s["dn"] = (*_w4(g, (E, H), I, c["G"]), I, c["G"])
    if c["delta"]:
        s["dgu"] = _normal(g, (T * k, 2 * I), 0.3)
        s["ddn"] = _normal(g, (T * k, H), 0.1)
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    return _library(state) if own else _plain(state)


def _library(s):
    import moe_lora_virtual_gb300 as mol

    c = s["c"]
    if c["op"] == "norm":
        return mol.mol_block_norm(s["y"], s["residual"], s["pre"], post_weight=s["post"],
                                  gate=s["gate"], residual_scale=s["scale"], eps=EPS)
    if c["op"] == "route":
        return mol.mol_moe_route(s["logits"], s["k"], renormalize=s["renorm"], scale=s["scale"])
    if c["op"] == "linear":
        return mol.mol_w4_linear(s["x"], mol.W4(*s["w"]))
    gu, dn = s["gu"], s["dn"]
    if c["fmt"] == "w4":
        gu, dn = mol.W4(*gu), mol.W4(*dn)
    if not c["delta"]:
        return mol.mol_moe_forward(s["x"], s["ids"], s["w"], gu, dn)
    act = mol.mol_moe_gate_up(s["x"], s["ids"], gu, delta=s["dgu"])
    return mol.mol_moe_down(act, s["ids"], s["w"], dn, delta=s["ddn"])


def _decode(w, rows=None):
    """fp32 values [..., K] of 4-bit rows (of rows[...] along the first axis)."""
    q, sc, K, G = w
    if rows is not None:
        q, sc = q[rows], sc[rows]
    lead = q.shape[:-1]
    words = q.contiguous().view(torch.int32).view(*lead, -1, 4, 4)  # block, t, i
    j = torch.arange(8, device=q.device, dtype=torch.int32)
    shift = torch.where(j % 2 == 0, j * 2, 16 + (j - 1) * 2)
    v = (words.transpose(-1, -2).unsqueeze(-1) >> shift) & 15       # block, i, t, j
    v = (v.to(torch.float32) - 8).reshape(*lead, -1, G) * sc.to(torch.float32).unsqueeze(-1)
    return v.reshape(*lead, -1)[..., :K]


def _rms(v, w):
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * w.to(torch.float32)


def _plain(s):
    c = s["c"]
    if c["op"] == "norm":
        y = s["y"].to(torch.float32)
        if s["post"] is not None:
            y = _rms(y, s["post"])
        if s["gate"] is not None:
            y = y * s["gate"].to(torch.float32)
        r = s["residual"].to(torch.float32) + s["scale"] * y
        return r.to(torch.bfloat16), _rms(r, s["pre"]).to(torch.bfloat16)
    if c["op"] == "route":
        v = s["logits"].to(torch.float32)
        T, E = v.shape
        e = torch.arange(E, device=v.device)
        a, b = v.unsqueeze(2), v.unsqueeze(1)
        ahead = (b > a) | ((b == a) & (e.view(1, 1, E) < e.view(1, E, 1)))
        rank = ahead.sum(2)
        ids = torch.zeros(T, E, dtype=torch.int64, device=v.device).scatter_(
            1, rank, e.expand(T, E))[:, :s["k"]]
        top = v.gather(1, ids)
        high = top[:, :1]
        p = torch.where(top == -math.inf, 0.0, torch.exp(top - high))
        total = (p if s["renorm"] else
                 torch.where(v == -math.inf, 0.0, torch.exp(v - high))).sum(1, keepdim=True)
        ids = torch.where(top == -math.inf, -1, ids).to(torch.int32)
        return ids, torch.where(ids < 0, 0.0, p * s["scale"] / total)
    if c["op"] == "linear":
        return (s["x"].to(torch.float32) @ _decode(s["w"]).T).to(torch.bfloat16)
    T, k, H, I = c["T"], c["k"], c["H"], c["I"]
    ids = s["ids"].reshape(-1).to(torch.int64)
    at = ids.clamp(min=0)
    deq = _decode if c["fmt"] == "w4" else lambda w, rows: w[rows].to(torch.float32)
    x = s["x"].to(torch.float32).repeat_interleave(k, 0).unsqueeze(-1)
    v = torch.bmm(deq(s["gu"], at), x).squeeze(-1)
    if c["delta"]:
        v = v + s["dgu"].to(torch.float32)
    gate, up = v[:, :I], v[:, I:]
    act = gate / (1 + torch.exp(-gate)) * up
    out = torch.bmm(deq(s["dn"], at), act.unsqueeze(-1)).squeeze(-1)
    if c["delta"]:
        out = out + s["ddn"].to(torch.float32)
    out = torch.where((ids >= 0).unsqueeze(1), out * s["w"].view(-1, 1), 0.0)
    return out.view(T, k, H).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------------- what it takes
def _active(c):
    """Experts that get a token, on average."""
    keep = 1 - c["drop"]
    p = (c["k"] - c["hot"]) / (c["E"] - c["hot"])
    return (c["hot"] * (1 - c["drop"] ** c["T"])
            + (c["E"] - c["hot"]) * (1 - (1 - p * keep) ** c["T"]))


def work(case):
    c, T = case, case["T"]
    if c["op"] == "norm":
        H = c["H"]
        rows = 4 + (c["gate"] == "token")
        vecs = 1 + (c["gate"] == "row") + c["post"]
        return dict(bytes=2.0 * H * (T * rows + vecs), flops=10.0 * T * H)
    if c["op"] == "route":
        return dict(bytes=T * (c["E"] * (4.0 if c["dtype"] == "f32" else 2.0) + 8.0 * c["k"]),
                    flops=4.0 * T * c["E"])
    if c["op"] == "linear":
        w = c["N"] * c["K"] * (0.5 + 2.0 / c["G"])
        return dict(bytes=w + 2.0 * T * (c["K"] + c["N"]), flops=2.0 * T * c["N"] * c["K"])
    k, H, I = c["k"], c["H"], c["I"]
    pairs = T * k * (1 - c["drop"])
    b = _active(c) * _expert_bytes(c) + 4.0 * T * H + 8.0 * T * k
    if c["delta"]:
        b += pairs * 2.0 * (2 * I + H)
    return dict(bytes=b, flops=2.0 * pairs * 3 * H * I)


# --------------------------------------------------------------------------------------- 64 bits
def _values64(w, e):
    """Expert (or row block) e's 4-bit rows as float64 [rows, K], nibble by nibble."""
    q, sc, K, G = w
    q, sc = (q, sc) if e is None else (q[e], sc[e])
    n, Kp = q.shape[0], q.shape[1] * 2
    low, high = (q & 15), (q >> 4)
    # input i of a block of 128: byte and half of it
    at = []
    for i in range(128):
        word = 4 * (i % 32 // 8) + i // 32
        nib = (i % 8) // 2 + 4 * (i % 2)
        at.append(word * 8 + nib)
    at = torch.tensor(at, device=q.device)
    nibbles = torch.stack([low, high], -1).view(n, Kp // 128, 128)
    out = nibbles[:, :, at].reshape(n, Kp).double() - 8.0
    return (out * sc.double().repeat_interleave(G, 1))[:, :K]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        y, r = s["y"].double(), s["residual"].double()
        if s["post"] is not None:
            y = y / torch.sqrt((y ** 2).sum(1, keepdim=True) / c["H"] + EPS) * s["post"].double()
        if s["gate"] is not None:
            y = y * s["gate"].double()
        r = r + s["scale"] * y
        return r, r / torch.sqrt((r ** 2).sum(1, keepdim=True) / c["H"] + EPS) * s["pre"].double()
    if c["op"] == "route":
        v = s["logits"].double()
        val, ids = torch.sort(v, dim=1, descending=True, stable=True)
        val, ids = val[:, :c["k"]], ids[:, :c["k"]]
        none = torch.isneginf(val)
        p = torch.softmax(val if c["renorm"] else v, 1)
        p = p if c["renorm"] else p.gather(1, ids)
        p = torch.where(none, 0.0, p * s["scale"])
        return None, p
    if c["op"] == "linear":
        return s["x"].double() @ _values64(s["w"], None).T
    I = c["I"]
    x, out = s["x"].double(), torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for e in sorted(set(s["ids"].view(-1).tolist()) - {-1}):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        pair = t * c["k"] + j
        gu, dn = ((_values64(s["gu"], e), _values64(s["dn"], e)) if c["fmt"] == "w4"
                  else (s["gu"][e].double(), s["dn"][e].double()))
        v = x[t] @ gu.T
        if c["delta"]:
            v = v + s["dgu"][pair].double()
        h = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]
        d = h @ dn.T
        if c["delta"]:
            d = d + s["ddn"][pair].double()
        out.index_add_(0, t, d * s["w"][t, j].double().unsqueeze(1))
    return out
