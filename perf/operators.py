"""Cases of the 4-bit weight operators: matrix-vector products (`moe_w4_matvec`) and
the whole mixture-of-experts layer for a few tokens (`moe_w4_forward`).

A weight tensor [.., N, K] is held as codes uint8 [.., N, K/2] (even k in the low
nibble), scales [.., N, ceil(K/group)] in fp32 or bf16 and, optionally, zero points
uint8 of the scales' shape (8 without them); it stands for scale * (code - zero).
"""
import numpy as np
import torch

own = False

SCALES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    def mv(name, T, K, N, group, scale, zeros, out):
        return dict(name=name, op="matvec", T=T, K=K, N=N, group=group, scale=scale, zeros=zeros,
                    out=out)

    def layer(name, T, H, I, E, k, group, scale, zeros, zipf=False, renorm=True):
        return dict(name=name, op="layer", T=T, H=H, I=I, E=E, k=k, group=group, scale=scale,
                    zeros=zeros, zipf=zipf, renorm=renorm)

    return [
        # one token through a small projection: launch and load latency
        mv("mv_t1_2048x2048", 1, 2048, 2048, 128, "bf16", False, "bf16"),
        # one token through the gate/up width of a dense layer: streaming rate
        mv("mv_t1_4096x28672", 1, 4096, 28672, 128, "bf16", False, "bf16"),
        # a small decode batch through a down projection (long K), zero points
        mv("mv_t8_14336x4096", 8, 14336, 4096, 64, "fp32", True, "bf16"),
        # odd rows and a short last group, fp32 logits out
        mv("mv_t5_7200x1027", 5, 7200, 1027, 128, "fp32", False, "fp32"),
        # the widest decode batch, the finest groups
        mv("mv_t64_7168x4096", 64, 7168, 4096, 32, "bf16", True, "bf16"),
        # a tiny layer of odd sizes, weights not renormalised
        layer("layer_tiny_t3", 3, 416, 224, 5, 3, 32, "fp32", True, renorm=False),
        # fine-grained experts: one token (latency), a small batch, a full one
        layer("layer_e128_t1", 1, 2048, 768, 128, 8, 128, "bf16", False),
        layer("layer_e128_t16", 16, 2048, 768, 128, 8, 64, "bf16", True),
        # eight large experts: one token (two experts), and 64 (all of them)
        layer("layer_e8_t1", 1, 4096, 14336, 8, 2, 128, "bf16", False),
        layer("layer_e8_t64", 64, 4096, 14336, 8, 2, 128, "fp32", False),
        # many experts with skewed popularity
        layer("layer_e256_t8", 8, 7168, 2048, 256, 8, 128, "bf16", False, zipf=True),
        layer("layer_e256_t32", 32, 7168, 2048, 256, 8, 128, "bf16", True, zipf=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _uneven(rng, lo, hi, units):
    """A size in lo..hi (over its logarithm): an odd multiple of one of `units`."""
    unit = rng.choice([u for u in units if u <= hi])
    return unit * (max(0, _log(rng, max(lo, unit), hi) // unit - 1) // 2 * 2 + 1)


def draw(rng):
    case = dict(group=rng.choice((32, 64, 128)), scale=rng.choice(("fp32", "bf16")),
                zeros=rng.random() < 0.5, T=_log(rng, 1, 64))
    if rng.random() < 0.5:
        K = _uneven(rng, 32, 14400, (32, 128))
        N = _uneven(rng, 1, min(30000, (1 << 27) // K), (1, 16))
        return dict(case, op="matvec", K=K, N=N, out=rng.choice(("bf16", "fp32")))
    E = _log(rng, 1, 256)
    H = _uneven(rng, 128, 7200, (32, 128))
    I = _uneven(rng, 64, min(14400, (1 << 30) // (3 * H * E)), (32, 128))
    return dict(case, op="layer", H=H, I=I, E=E, k=rng.randint(1, min(8, E)),
                zipf=rng.random() < 0.5, renorm=rng.random() < 0.75)


# ---------------------------------------------------------------- inputs


def _codes(g, *shape):
    """Bell-shaped codes around 8, as a quantiser leaves them: the mean of two nibbles."""
    dev = g.device
    a = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device=dev)
    b = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device=dev)
    lo = ((a & 15) + (b & 15) + 1) >> 1
    hi = ((a >> 4) + (b >> 4) + 1) >> 1
    return lo | (hi << 4)


def _weight(g, case, *shape):
    rows, K = shape[:-1], shape[-1]
    groups = -(-K // case["group"])
    codes = _codes(g, *rows, K // 2)
    scales = (0.005 + 0.01 * torch.rand(*rows, groups, generator=g, device=g.device))
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(5, 12, (*rows, groups), generator=g, dtype=torch.uint8,
                              device=g.device)
    return dict(codes=codes, scales=scales.to(SCALES[case["scale"]]), zeros=zeros)


def _logit_bias(case):
    """Expert popularity of the skewed cases: 2 log p, p falling as rank^-1.1."""
    p = np.arange(1, case["E"] + 1, dtype=np.float64) ** -1.1
    return 2.0 * np.log(p / p.sum()) if case["zipf"] else np.zeros(case["E"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, s = case["T"], dict(case)
    if case["op"] == "matvec":
        s["x"] = torch.randn(T, case["K"], generator=g, device="cuda").to(torch.bfloat16)
        s["w"] = _weight(g, case, case["N"], case["K"])
    else:
        E, H, I = case["E"], case["H"], case["I"]
        bias = torch.from_numpy(_logit_bias(case)).float().cuda()
        s["logits"] = torch.randn(T, E, generator=g, device="cuda") + bias
        s["x"] = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        s["w13"] = _weight(g, case, E, 2 * I, H)
        s["w2"] = _weight(g, case, E, H, I)
    if own:
        import mixture_experts_layer_align_gb300 as moe

        def handle(w):
            return moe.W4Tensor(w["codes"], w["scales"], w["zeros"], group=case["group"])

        s["moe"] = moe
        if case["op"] == "matvec":
            s["w"] = handle(s["w"])
            s["y"] = torch.empty(T, case["N"], dtype=_out_dtype(case), device="cuda")
        else:
            s["w13"], s["w2"] = handle(s["w13"]), handle(s["w2"])
            s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
            s["ids"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty(T, case["k"], dtype=torch.float32, device="cuda")
            s["workspace"] = moe.alloc_w4_workspace(T, H, I, E, case["k"])
    return s


def _out_dtype(case):
    return torch.float32 if case.get("out") == "fp32" else torch.bfloat16


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        if s["op"] == "matvec":
            return s["moe"].moe_w4_matvec(s["x"], s["w"], out=s["y"])
        out = s["moe"].moe_w4_forward(s["x"], s["logits"], s["w13"], s["w2"], s["k"],
                                      renormalize=s["renorm"], out=s["out"],
                                      workspace=s["workspace"], topk_ids_out=s["ids"],
                                      topk_w_out=s["weights"])
        return dict(out=out, ids=s["ids"], weights=s["weights"])
    if s["op"] == "matvec":
        return (s["x"].float() @ _values(s["w"], s["group"]).T).to(_out_dtype(s))
    return _plain_layer(s)


def _values(w, group, rows=None):
    """fp32 values of a weight tensor, or of the first-axis entries `rows` of it."""
    codes, scales, zeros = ((t if t is None or rows is None else t[rows])
                            for t in (w["codes"], w["scales"], w["zeros"]))
    K = 2 * codes.shape[-1]
    v = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()

    def spread(t):
        return t.float().repeat_interleave(group, dim=-1)[..., :K]

    v -= 8.0 if zeros is None else spread(zeros)
    v *= spread(scales)
    return v


def _silu_product(gate_up, I):
    gate, up = gate_up[..., :I], gate_up[..., I:]
    return gate / (1 + torch.exp(-gate)) * up


def _plain_layer(s):
    T, E, I, k = s["T"], s["E"], s["I"], s["k"]
    x = s["x"].float()
    logits = s["logits"]
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = e.gather(1, ids)
    weights = chosen / (chosen if s["renorm"] else e).sum(dim=1, keepdim=True)
    if T * k <= E:  # each pair's own copy of its expert
        rows = ids.reshape(-1)
        xp = x.repeat_interleave(k, dim=0).unsqueeze(-1)
        h = _silu_product((_values(s["w13"], s["group"], rows) @ xp).squeeze(-1), I)
        y = (_values(s["w2"], s["group"], rows) @ h.unsqueeze(-1)).reshape(T, k, -1)
    else:  # every expert on every token, then each token's own
        h = _silu_product(x @ _values(s["w13"], s["group"]).transpose(1, 2), I)
        y = h @ _values(s["w2"], s["group"]).transpose(1, 2)
        y = y[ids, torch.arange(T, device=x.device)[:, None]]
    out = (weights.unsqueeze(-1) * y).sum(dim=1).to(torch.bfloat16)
    return dict(out=out, ids=ids.to(torch.int32), weights=weights)


# ---------------------------------------------------------------- figures


def _touched(case):
    """Mean number of experts that T tokens choose (logits as prepare() draws them)."""
    rng = np.random.default_rng(1)
    bias, counts = _logit_bias(case), []
    for _ in range(20):
        l = rng.standard_normal((case["T"], case["E"])) + bias
        counts.append(len(np.unique(np.argsort(-l, axis=1)[:, :case["k"]])))
    return float(np.mean(counts))


def work(case):
    T = case["T"]

    def tensor(N, K):
        per_group = (4 if case["scale"] == "fp32" else 2) + (1 if case["zeros"] else 0)
        return N * K / 2 + N * -(-K // case["group"]) * per_group

    if case["op"] == "matvec":
        K, N = case["K"], case["N"]
        return {"bytes": tensor(N, K) + 2 * T * K + (4 if case["out"] == "fp32" else 2) * T * N,
                "flops": 2 * T * N * K}
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    return {"bytes": _touched(case) * (tensor(2 * I, H) + tensor(H, I)) + 4 * T * H + 4 * T * E
            + 8 * T * k,
            "flops": 6 * T * k * H * I}


def exact(case, seed):
    """The definitions in fp64, expert by expert over the tokens that chose it."""
    s = prepare_plain(case, seed)
    x = s["x"].double()

    def matrix(w, at=()):
        q = w["codes"][at].to(torch.int16)
        v = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
        v[:, 0::2], v[:, 1::2] = (q % 16).double(), (q // 16).double()
        group = torch.arange(v.shape[1], device=q.device) // case["group"]
        zero = w["zeros"][at].double()[:, group] if case["zeros"] else 8.0
        return (v - zero) * w["scales"][at].double()[:, group]

    if case["op"] == "matvec":
        return x @ matrix(s["w"]).T
    logits = s["logits"].double().cpu().numpy()
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :case["k"]]
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    weights = np.take_along_axis(p, ids, axis=1)
    if case["renorm"]:
        weights /= weights.sum(axis=1, keepdims=True)
    out = torch.zeros_like(x)
    for expert in np.unique(ids):
        t, j = np.nonzero(ids == expert)
        tok = torch.from_numpy(t).to(x.device)
        gate, up = (x[tok] @ matrix(s["w13"], int(expert)).T).split(case["I"], dim=1)
        y = (gate * torch.sigmoid(gate) * up) @ matrix(s["w2"], int(expert)).T
        out[tok] += torch.from_numpy(weights[t, j]).to(x.device)[:, None] * y
    return dict(out=out, ids=torch.from_numpy(ids.astype(np.int32)),
                weights=torch.from_numpy(weights))


def prepare_plain(case, seed):
    """prepare()'s inputs as plain tensors, whichever side asks."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
