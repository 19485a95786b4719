"""Measured cases of the adapter operators: a W4A16 projection with low-rank
adapters of many requests beside it, its gradients, and the AdamW step over
the adapters' tensors.

``run`` computes a case in its plain form (elementary torch operations in
32 bits, rounded once at the end), or, where ``own`` is true, with the
framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
NIBBLE_OF_K = (0, 4, 1, 5, 2, 6, 3, 7)  # nibble of a packed word that holds k-offset 0..7

# (K, N) of the fused projections of the two model families in synth/configs.py
LLAMA = ((4096, 6144), (4096, 4096), (4096, 28672), (14336, 4096))
QWEN = ((2560, 6144), (4096, 2560), (2560, 19456), (9728, 2560))
FAMILIES = {"llama8b": LLAMA, "qwen3_4b": QWEN}


def listed():
    def lora(name, M, K, N, R, S, ids, dtype="bf16", group=128, sym=False, bias=False, save_u=False):
        return dict(name=name, op="lora", M=M, K=K, N=N, R=R, S=S, ids=ids, dtype=dtype, group=group, sym=sym,
                    bias=bias, save_u=save_u)

    def bwd(name, M, K, N, R, S, ids, dtype="bf16", group=128, sym=False):
        return dict(name=name, op="lora_bwd", M=M, K=K, N=N, R=R, S=S, ids=ids, dtype=dtype, group=group, sym=sym)

    def adamw(name, family, layers, rank, bits, param="f32", grad="bf16", copy="bf16", odd=False):
        return dict(name=name, op="adamw", family=family, layers=layers, rank=rank, bits=bits, param=param,
                    grad=grad, copy=copy, odd=odd)

    return [
        # one user's next token through the attention output projection: latency alone
        lora("decode_1", 1, 4096, 4096, 16, 8, "mixed"),
        # sixteen users decode together, nearly each with an adapter of their own
        lora("decode_16", 16, 4096, 6144, 16, 32, "mixed"),
        # five users, wide adapters, the long reduction of a down projection, fp16 with a bias
        lora("decode_5_down", 5, 9728, 2560, 64, 4, "mixed", dtype="f16", sym=True, bias=True),
        # an odd batch (decode steps and short prompts together), tokens of many requests in any order
        lora("batch_67", 67, 2560, 19456, 32, 16, "mixed", dtype="f16", group=64, sym=True),
        # a prefill step of several requests, one after another, through gate + up
        lora("prefill_1920", 1920, 4096, 28672, 16, 6, "runs"),
        # the forward pass of a training step: one wide adapter, u kept for the backward pass
        lora("train_fwd_1920", 1920, 14336, 4096, 64, 1, "one", save_u=True),
        # a small training step's gradients through one square projection
        bwd("bwd_128", 128, 4096, 4096, 16, 1, "one"),
        # an odd number of tokens of three adapters trained side by side, fp16, small groups
        bwd("bwd_1921", 1921, 4096, 6144, 16, 3, "runs", dtype="f16", group=64),
        # the largest projection's gradients with a wide adapter
        bwd("bwd_wide_1920", 1920, 4096, 28672, 64, 1, "one"),
        # one layer's adapters with odd-sized tensors beside them: launch latency
        adamw("adamw_layer_8bit", "qwen3_4b", 1, 16, 8, odd=True),
        # every adapter tensor of a model (256 tensors), states in 32 bits
        adamw("adamw_model_32bit", "llama8b", 32, 16, 32),
        # the same model with wide adapters, states in 8 bits: memory rate
        adamw("adamw_model_8bit", "llama8b", 32, 64, 8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("lora", "lora", "lora_bwd", "adamw"))
    if op == "adamw":
        bits = rng.choice((8, 32))
        param = rng.choice(("f32", "f32", "bf16", "f16"))
        return dict(op=op, family=rng.choice(tuple(FAMILIES)), layers=_log(rng, 1, 32), rank=rng.choice((8, 16, 24, 32, 64)),
                    bits=bits, param=param, grad=rng.choice(("f32", "bf16", "f16")) if param == "f32" else param,
                    copy=rng.choice(("none", "bf16", "f16")) if param == "f32" else "none", odd=rng.random() < 0.5)
    group = rng.choice((32, 64, 128, 128))
    K = group * max(1, _log(rng, 256, 14336) // group)  # ragged last runs of 128 k among them
    sym = rng.random() < 0.5
    N = _log(rng, 64, 8192)
    if not sym:  # packed zero points come eight rows to a word
        N = (N + 7) // 8 * 8
    S = _log(rng, 1, 48)
    R = rng.choice((8, 16, 24, 32, 64, 128)) if S <= 16 else rng.choice((8, 16, 32))
    case = dict(op=op, M=_log(rng, 1, 2048) if op == "lora" else _log(rng, 16, 2048), K=K, N=N, R=R, S=S,
                ids=rng.choice(("one", "runs", "mixed")), dtype=rng.choice(("f16", "bf16")), group=group, sym=sym)
    if op == "lora":
        case["bias"] = rng.random() < 0.3
        case["save_u"] = rng.random() < 0.3
    return case


# ------------------------------------------------------------- inputs ---

def _adamw_sizes(case):
    sizes = []
    for _ in range(case["layers"]):
        for K, N in FAMILIES[case["family"]]:
            sizes += [case["rank"] * K, N * case["rank"]]
    if case["odd"]:
        sizes += [1, 255, 257, 2559, 12345]
    return sizes


def _prepare_adamw(case, gen, dev):
    # tensors are views of flat buffers, each starting at a multiple of 256
    sizes = _adamw_sizes(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += (n + 255) // 256 * 256
    real = torch.zeros(total, dtype=torch.bool, device=dev)
    for s, n in zip(starts, sizes):
        real[s:s + n] = True
    normal = lambda k: torch.randn(total, generator=gen, device=dev).mul_(k)  # noqa: E731
    p = (normal(0.02) * real).to(DTYPES[case["param"]])
    # gradients of tensors of one model differ by orders of magnitude between and inside tensors
    g = (normal(1e-3) * torch.exp(normal(1.0)) * real).to(DTYPES[case["grad"]])
    m = normal(3e-4) * torch.exp(normal(1.0)) * real
    v = (m * m + torch.square(normal(5e-4))) * real
    state = dict(case=case, starts=starts, sizes=sizes, p=p, g=g,
                 hyper=dict(lr=2e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=100, grad_scale=0.5,
                            seed=int(torch.randint(0, 1 << 31, (1,), generator=gen, device=dev))))
    if case["copy"] != "none":
        state["copy"] = p.to(DTYPES[case["copy"]])
    if case["bits"] == 32:
        state |= dict(m=m, v=v)
    else:
        # codes of the blocks of 256 with their scales, and room for the moments that they stand for
        ms, rs = m.view(-1, 256).abs().amax(1), torch.sqrt(v).view(-1, 256).amax(1)
        cm = (127 * torch.sqrt(m.view(-1, 256).abs() / ms[:, None].clamp(min=1e-30))).round().nan_to_num() * torch.sign(m.view(-1, 256))
        cv = (255 * torch.sqrt(torch.sqrt(v).view(-1, 256) / rs[:, None].clamp(min=1e-30))).round().nan_to_num()
        state |= dict(m=cm.to(torch.int8).view(-1), v=cv.to(torch.uint8).view(-1), ms=ms, rs=rs,
                      m32=torch.empty_like(m), v32=torch.empty_like(v))
    if own:
        # the step's table of tensors: the handle that a training program lays out once (the data are the same)
        import int4_weight_only_linear_amd as L
        cut = lambda t, per=1: [t[a // per:(a + n + per - 1) // per] for a, n in zip(starts, sizes)]  # noqa: E731
        eight = case["bits"] == 8
        state["plan"] = L.w4a16_adamw_plan(
            cut(p), cut(g), cut(state["m"]), cut(state["v"]), m_scales=cut(state["ms"], 256) if eight else None,
            v_scales=cut(state["rs"], 256) if eight else None, copies=cut(state["copy"]) if "copy" in state else None)
    return state


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen, dev)
    dt = DTYPES[case["dtype"]]
    M, K, N, R, S, G = case["M"], case["K"], case["N"], case["R"], case["S"], case["K"] // case["group"]
    normal = lambda shape, k: torch.randn(shape, generator=gen, device=dev).mul_(k).to(dt)  # noqa: E731
    words = lambda shape: torch.randint(-(1 << 31), 1 << 31, shape, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)  # noqa: E731
    ids = torch.zeros(M, dtype=torch.int64, device=dev)
    if case["ids"] != "one":
        ids = torch.randint(0, S, (M,), generator=gen, device=dev)
        # about one token in eight belongs to a request without an adapter
        ids[torch.rand(M, generator=gen, device=dev) < 0.125] = -1
        if case["ids"] == "runs":
            # the requests' tokens one request after another, in a drawn order
            ids = torch.sort(ids).values
            order = torch.argsort(torch.rand(S + 1, generator=gen, device=dev))
            ids = ids[torch.argsort(order[ids + 1], stable=True)]
    state = dict(
        case=case, x=normal((M, K), 1.0), wq=words((N, K // 8)),
        scales=(torch.randn((N, G), generator=gen, device=dev).mul_(0.02).abs_() + 1e-3).to(dt),
        zp=None if case["sym"] else words((N // 8, G)),
        la=normal((S, R, K), K ** -0.5), lb=normal((S, N, R), 2.0 * R ** -0.5), ids=ids.to(torch.int32),
        alpha=torch.rand(S, generator=gen, device=dev) * 2 + 1,
        bias=normal((N,), 0.1) if case.get("bias") else None)
    if case["op"] == "lora_bwd":
        state["dy"] = normal((M, N), 0.05)
        # what the forward pass kept: x . A^T of each token's own adapter, in 32 bits
        every = (state["x"].float() @ state["la"].float().view(S * R, K).T).view(M, S, R)
        pick = every.gather(1, ids.clamp(min=0).view(M, 1, 1).expand(M, 1, R)).view(M, R)
        state["u"] = pick * (ids >= 0).view(M, 1)
    return state


# --------------------------------------------------------- plain form ---

def _weights(s):
    """The projection's weights [N, K] in 32 bits."""
    wq, (N, J) = s["wq"], s["wq"].shape
    n = torch.arange(N, device=wq.device).view(N, 1)
    c = torch.arange(J, device=wq.device).view(1, J)  # slice of eight k
    runs, tail = J // 16, J % 16
    run, sl = c // 16, c % 16
    word = torch.where(run < runs, 16 * run + 4 * (sl % 4) + sl // 4, c)  # stored word of the row
    tile, row = n // 16, n % 16
    inside = tile * 16 * J + torch.where(
        run < runs, 256 * run + 4 * (16 * (sl % 4) + row) + sl // 4, 256 * runs + tail * row + (c - 16 * runs))
    at = torch.where((tile + 1) * 16 <= N, inside, n * J + word)
    w = wq.view(-1)[at].view(N, J, 1)
    shift = 4 * torch.tensor(NIBBLE_OF_K, device=wq.device, dtype=torch.int32)
    q = ((w >> shift) & 15).view(N, J * 8).float()
    G = s["scales"].shape[1]
    if s["zp"] is None:
        z = 8.0
    else:
        z = ((s["zp"].view(N // 8, 1, G) >> (4 * torch.arange(8, device=wq.device, dtype=torch.int32)).view(1, 8, 1)) & 15)
        z = z.reshape(N, G, 1).float()
    return ((q.view(N, G, -1) - z) * s["scales"].float().view(N, G, 1)).view(N, J * 8)


def _own_mask(s):
    """[M, S] in 32 bits: alpha where the adapter is the token's own, 0 elsewhere; and the same with 1."""
    S = s["la"].shape[0]
    own_ = (s["ids"].view(-1, 1) == torch.arange(S, device=s["ids"].device).view(1, S)).float()
    return own_ * s["alpha"].view(1, S), own_


def _plain_lora(s):
    case = s["case"]
    M, R, S, K = case["M"], case["R"], case["S"], case["K"]
    x = s["x"].float()
    scaled, one = _own_mask(s)
    every = (x @ s["la"].float().view(S * R, K).T).view(M, S, R)
    up = s["lb"].float().transpose(1, 2).reshape(S * R, -1)
    y = x @ _weights(s).T + (every * scaled.view(M, S, 1)).view(M, S * R) @ up
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(s["x"].dtype)
    return (y, (every * one.view(M, S, 1)).sum(1)) if case["save_u"] else y


def _plain_bwd(s):
    case = s["case"]
    M, R, S, K, N = case["M"], case["R"], case["S"], case["K"], case["N"]
    x, dy, dt = s["x"].float(), s["dy"].float(), s["x"].dtype
    scaled, _ = _own_mask(s)
    la, lb = s["la"].float().view(S * R, K), s["lb"].float().transpose(1, 2).reshape(S * R, N)
    g = ((dy @ lb.T).view(M, S, R) * scaled.view(M, S, 1)).view(M, S * R)
    u = (s["u"].view(M, 1, R) * scaled.view(M, S, 1)).view(M, S * R)
    dx = dy @ _weights(s) + g @ la
    dla = (g.T @ x).view(S, R, K)
    dlb = (u.T @ dy).view(S, R, N).transpose(1, 2)
    return dx.to(dt), dla.to(dt), dlb.contiguous().to(dt)


def _mix(c):
    """A 32-bit integer hash of the 32-bit integers in c (int64)."""
    c = c ^ (c >> 16)
    c = (c * 0x7FEB352D) & 0xFFFFFFFF
    c = c ^ (c >> 15)
    c = (c * 0x846CA68B) & 0xFFFFFFFF
    return c ^ (c >> 16)


def _adamw_constants(h):
    return dict(decay=1.0 - h["lr"] * h["weight_decay"], rate=h["lr"] / (1.0 - h["beta1"] ** h["step"]),
                root=1.0 / math.sqrt(1.0 - h["beta2"] ** h["step"]))


def _plain_adamw(s):
    h, k, eight = s["hyper"], _adamw_constants(s["hyper"]), s["case"]["bits"] == 8
    m, v = _moments_8bit(s) if eight else (s["m"], s["v"])
    g = s["g"].float() * h["grad_scale"]
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1.0 - h["beta2"])
    r = torch.sqrt(v)
    p = s["p"].float() * k["decay"] - (m / (r * k["root"] + h["eps"])) * k["rate"]
    s["p"].copy_(p)
    out = {"p": s["p"]}
    if "copy" in s:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return out | {"m": s["m"], "v": s["v"]}
    count = torch.arange(m.numel(), device=m.device) + h["seed"] * 0x9E3779B9
    dither = _mix(count & 0xFFFFFFFF)
    m, r = m.view(-1, 256), r.view(-1, 256)
    ms, rs = m.abs().amax(1), r.amax(1)
    inv = lambda t: torch.where(t > 2.0 ** -100, 1.0 / t, 0.0).view(-1, 1)  # noqa: E731
    cm = torch.floor(torch.sqrt(m.abs() * inv(ms)) * 127.0 + (dither & 0xFFFF).view(-1, 256).float() * 2.0 ** -16)
    cv = torch.floor(torch.sqrt(r * inv(rs)) * 255.0 + (dither >> 16).view(-1, 256).float() * 2.0 ** -16)
    cv = torch.where(r > 0, cv.clamp(min=1.0), cv)
    s["m"].copy_((torch.sign(m) * cm.clamp(max=127.0)).view(-1))
    s["v"].copy_(cv.clamp(max=255.0).view(-1))
    s["ms"].copy_(ms)
    s["rs"].copy_(rs)
    # the moments that the new codes stand for, in 32 bits
    m, v = _moments_8bit(s)
    s["m32"].copy_(m)
    s["v32"].copy_(v)
    return out | {"m": s["m32"], "v": s["v32"]}


def _moments_8bit(s):
    m = s["m"].view(-1, 256).float() * (1.0 / 127.0)
    r = s["v"].view(-1, 256).float() * (1.0 / 255.0)
    r = (r * r) * s["rs"].view(-1, 1)
    return ((m * m.abs()) * s["ms"].view(-1, 1)).view(-1), (r * r).view(-1)


# ----------------------------------------------------------------- run ---

def _own_adamw(s):
    import int4_weight_only_linear_amd as L
    case, h = s["case"], s["hyper"]
    L.w4a16_adamw_step(s["plan"], lr=h["lr"], betas=(h["beta1"], h["beta2"]), eps=h["eps"],
                       weight_decay=h["weight_decay"], step=h["step"], grad_scale=h["grad_scale"], seed=h["seed"])
    out = {"p": s["p"]} | ({"copy": s["copy"]} if "copy" in s else {})
    if case["bits"] == 32:
        return out | {"m": s["m"], "v": s["v"]}
    L.w4a16_adamw_moments(s["plan"], s["m32"], s["v32"])  # what the codes stand for
    return out | {"m": s["m32"], "v": s["v32"]}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"lora": _plain_lora, "lora_bwd": _plain_bwd, "adamw": _plain_adamw}[op](s)
    if op == "adamw":
        return _own_adamw(s)
    import int4_weight_only_linear_amd as L
    group = s["case"]["group"]
    if op == "lora":
        return L.w4a16_lora_linear(s["x"], s["wq"], s["scales"], s["la"], s["lb"], s["ids"], s["zp"], s["bias"],
                                   s["alpha"], group_size=group, save_u=s["case"]["save_u"])
    return L.w4a16_lora_backward(s["dy"], s["x"], s["u"], s["wq"], s["scales"], s["la"], s["lb"], s["ids"], s["zp"],
                                 s["alpha"], group_size=group)


# ---------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "adamw":
        n = sum(_adamw_sizes(case))
        size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
        # 8 bits: codes and scales in and out, and the moments in 32 bits out
        state = 16 if case["bits"] == 32 else 4 + 16 / 256 + 8
        return {"bytes": n * (2 * size[case["param"]] + size[case["grad"]] + size[case["copy"]] + state), "flops": 20 * n}
    M, K, N, R, S, G = case["M"], case["K"], case["N"], case["R"], case["S"], case["K"] // case["group"]
    weights = N * K // 2 + 2 * N * G + (0 if case["sym"] else N * G // 2)
    # adapters that the tokens can name at most; each is read once
    used = 1 if case["ids"] == "one" else min(S, M)
    adapters = used * R * (K + N) * 2
    dense, low = 2 * M * N * K, 2 * M * R * (K + N)
    if case["op"] == "lora":
        return {"bytes": weights + adapters + 2 * M * (K + N) + 4 * M + (2 * N if case["bias"] else 0)
                + (4 * M * R if case["save_u"] else 0), "flops": dense + low}
    return {"bytes": weights + adapters + S * R * (K + N) * 2 + 2 * M * (2 * K + N) + 4 * M * (1 + R),
            "flops": dense + 2 * low}


# --------------------------------------------------------------- exact ---

def _exact_weights(s):
    """[N, K] in 64 bits, walking the stored words in order: row and slice of each from its place."""
    wq, (N, J) = s["wq"], s["wq"].shape
    i = torch.arange(N * J, device=wq.device)
    tile, off = i // (16 * J), i % (16 * J)
    whole = tile < N // 16
    runs, tail = J // 16, J % 16
    piece, e = (off % 256) // 4, off % 4
    block = off < 256 * runs
    rest = off - 256 * runs
    per = max(tail, 1)
    row_whole = tile * 16 + torch.where(block, piece % 16, rest // per)
    slice_whole = torch.where(block, off // 256 * 16 + 4 * e + piece // 16, 16 * runs + rest % per)
    j = i % J
    p = j % 16
    slice_last = torch.where(j // 16 < runs, j - p + 4 * (p % 4) + p // 4, j)
    row, sl = torch.where(whole, row_whole, i // J), torch.where(whole, slice_whole, slice_last)
    word = wq.reshape(-1).to(torch.int64) & 0xFFFFFFFF
    q = torch.empty((N, J * 8), dtype=torch.float64, device=wq.device)
    for k, t in enumerate(NIBBLE_OF_K):
        q[row, sl * 8 + k] = ((word >> (4 * t)) & 15).double()
    G = s["scales"].shape[1]
    z = torch.full((N, G), 8.0, dtype=torch.float64, device=wq.device)
    if s["zp"] is not None:
        for b in range(8):
            z[b::8] = (((s["zp"].to(torch.int64) & 0xFFFFFFFF) >> (4 * b)) & 15).double()
    size = J * 8 // G
    return (q - z.repeat_interleave(size, 1)) * s["scales"].double().repeat_interleave(size, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    W = _exact_weights(s)
    x = s["x"].double()
    M, R, S = case["M"], case["R"], case["S"]
    if case["op"] == "lora":
        y = x @ W.T
        u = torch.zeros((M, R), dtype=torch.float64, device=x.device)
        for a in range(S):
            rows = torch.nonzero(s["ids"] == a).view(-1)
            if len(rows):
                u[rows] = x[rows] @ s["la"][a].double().T
                y[rows] += float(s["alpha"][a]) * (u[rows] @ s["lb"][a].double().T)
        if s["bias"] is not None:
            y += s["bias"].double()
        return (y, u) if case["save_u"] else y
    dy, u = s["dy"].double(), s["u"].double()
    dx = dy @ W
    dla, dlb = torch.zeros_like(s["la"], dtype=torch.float64), torch.zeros_like(s["lb"], dtype=torch.float64)
    for a in range(S):
        rows = torch.nonzero(s["ids"] == a).view(-1)
        if len(rows):
            k = float(s["alpha"][a])
            g = k * (dy[rows] @ s["lb"][a].double())
            dx[rows] += g @ s["la"][a].double()
            dla[a] = g.T @ x[rows]
            dlb[a] = k * (dy[rows].T @ u[rows])
    return dx, dla, dlb


def _exact_adamw(s):
    h, eight = s["hyper"], s["case"]["bits"] == 8
    g = s["g"].double() * h["grad_scale"]
    if eight:
        spread = lambda t: t.double().repeat_interleave(256)  # noqa: E731
        c = s["m"].double() / 127
        m = torch.sign(c) * c ** 2 * spread(s["ms"])
        v = (s["v"].double() / 255) ** 4 * spread(s["rs"]) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    mh, vh = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p = s["p"].double()
    p = p - h["lr"] * (mh / (vh ** 0.5 + h["eps"]) + h["weight_decay"] * p)
    out = {"p": p} | ({"copy": p} if "copy" in s else {})
    if not eight:
        return out | {"m": m, "v": v}
    # the codes: power laws of the share of the block's largest, rounded up or down by the dither
    lane = torch.arange(m.numel(), device=m.device)
    d = (lane + h["seed"] * 0x9E3779B9) % (1 << 32)
    for down, by in ((16, 2146121005), (15, 2221713035), (16, 1)):  # two rounds of shift, exclusive or, product
        d = ((d ^ (d // (1 << down))) * by) % (1 << 32)
    low, high = (d % 65536).double() / 65536, (d // 65536).double() / 65536
    top_m, top_r = (t.view(-1, 256).amax(1).repeat_interleave(256) for t in (m.abs(), v ** 0.5))
    part = lambda a, b: torch.where(b > 0, a / b.clamp(min=1e-300), 0.0)  # noqa: E731
    cm = (127 * part(m.abs(), top_m) ** 0.5 + low).floor().clamp(max=127)
    cv = (255 * part(v ** 0.5, top_r) ** 0.5 + high).floor().clamp(max=255)
    cv = torch.where(v > 0, cv.clamp(min=1), cv)
    return out | {"m": torch.sign(m) * (cm / 127) ** 2 * top_m, "v": (cv / 255) ** 4 * top_r ** 2}
