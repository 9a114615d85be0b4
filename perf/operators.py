"""What the token-block operators cost: lookups with their gradient, dropout,
the residual's addition with a root-mean-square norm, and products grouped by
expert. For each case: its inputs, one pass (in plain torch operations, or
through the library's entry points), the least it has to move and compute,
and its result in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}


def listed():
    return [
        # one request: the last 48 ids of a user's history, 128-wide rows as in the large configuration
        dict(name="lookup_request", op="lookup", n=48, rows=1_000_000, d=128, table="bf16", out="bf16"),
        # a training batch of 64-id histories into 1,024-wide rows
        dict(name="lookup_batch", op="lookup", n=65_536, rows=400_000, d=1024, table="bf16", out="bf16"),
        # its gradient: skewed ids, a dense fp32 gradient of the whole table
        dict(name="lookup_gradient", op="lookup_grad", n=65_536, rows=100_000, d=512, grad="bf16", table="f32"),
        # one token through a serving block: residual, norm, 8-bit rows for the experts
        dict(name="norm_token", op="norm", rows=4, d=2048, x="bf16", y="e4m3", residual=True),
        # a prompt or a training batch through the same, with what the backward pass keeps
        dict(name="norm_batch", op="norm", rows=16_384, d=4096, x="bf16", y="e4m3", residual=True),
        # the backward pass of an fp16 norm, a width that is no power of two
        dict(name="norm_gradient", op="norm_grad", rows=20_000, d=2040, x="f16", residual=True),
        # a hidden layer of the medium configuration in training
        dict(name="dropout_layer", op="dropout", n=2048 * 512, x="f32", p=0.1, residual=False),
        # a residual branch of a training batch
        dict(name="dropout_branch", op="dropout", n=32_768 * 1024, x="bf16", p=0.25, residual=True),
        # 12 routed rows of single tokens: weights are all there is to read
        dict(name="experts_token", op="experts", M=12, spare=4, E=8, N=4096, K=1024, x="bf16", y="bf16", relu=True),
        # the top layers' odd width, ragged experts, fp16, ReLU
        dict(name="experts_ragged", op="experts", M=20_000, spare=480, E=24, N=1024, K=479, x="f16", y="f16", relu=True),
        # a prompt in 8 bits
        dict(name="experts_8bit", op="experts", M=16_384, spare=0, E=16, N=4096, K=2048, x="e4m3", y="bf16", relu=False),
        # the backward pass of a training batch: three gradients
        dict(name="experts_gradient", op="experts_grad", M=16_384, spare=100, E=8, N=4096, K=1024, x="bf16", dw="f32",
             relu=True),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "norm", "norm_grad", "dropout", "experts", "experts", "experts_grad"])
    if op == "lookup":
        d = _between(rng, 16, 1024) if rng.random() < 0.4 else 8 * _between(rng, 2, 128)
        n = min(_between(rng, 16, 65_536), (65_536 * 1024) // d)
        return dict(op=op, n=n, rows=min(_between(rng, 1000, 1_000_000), 400_000_000 // d), d=d,
                    table=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]))
    if op == "lookup_grad":
        d = _between(rng, 16, 1024) if rng.random() < 0.4 else 8 * _between(rng, 2, 128)
        return dict(op=op, n=min(_between(rng, 16, 65_536), (65_536 * 512) // d),
                    rows=min(_between(rng, 100, 500_000), 51_200_000 // d), d=d,
                    grad=rng.choice(["f32", "bf16", "f16"]), table=rng.choice(["f32", "bf16", "f16"]))
    if op in ("norm", "norm_grad"):
        d = _between(rng, 64, 8192) if rng.random() < 0.4 else 16 * _between(rng, 4, 512)
        rows = min(_between(rng, 1, 32_768), (16_384 * 4096) // d)
        c = dict(op=op, rows=rows, d=d, x=rng.choice(["f32", "bf16", "f16"]), residual=rng.random() < 0.7)
        if op == "norm":
            c["y"] = rng.choice(["e4m3", c["x"]])
        return c
    if op == "dropout":
        return dict(op=op, n=_between(rng, 1000, 32_768 * 1024), x=rng.choice(["f32", "bf16", "f16"]),
                    p=rng.choice([0.05, 0.1, 0.2, 0.3, 0.5]), residual=rng.random() < 0.5)
    N = _between(rng, 64, 4096) if rng.random() < 0.4 else 16 * _between(rng, 4, 256)
    K = _between(rng, 64, 4096) if rng.random() < 0.4 else 16 * _between(rng, 4, 256)
    M = min(_between(rng, 1, 20_000), (16_384 * 4096 * 1024) // (N * K))
    E = min(_between(rng, 2, 64), 134_000_000 // (N * K))
    c = dict(op=op, M=M, spare=rng.choice([0, 0, 7, 100]), E=max(1, E), N=N, K=K, relu=rng.random() < 0.5)
    if op == "experts":
        c["x"] = rng.choice(["bf16", "f16", "e4m3"])
        c["y"] = rng.choice(["bf16", "f32"]) if c["x"] == "e4m3" else c["x"]
    else:
        c["x"] = rng.choice(["bf16", "f16"])
        c["dw"] = rng.choice(["f32", c["x"]])
    return c


# ------------------------------------------------------------------ inputs

def _ld(width, dt):
    """Elements from one row to the next: rows start on 16 bytes."""
    per = 16 // SIZE[dt]
    return (width + per - 1) // per * per


def _rows(g, rows, width, dt, scale=1.0, lead=()):
    """Normal values in rows that start on 16 bytes."""
    t = torch.randn((*lead, rows, width), generator=g, device="cuda") * scale
    buf = torch.zeros((*lead, rows, _ld(width, dt)), dtype=DT[dt], device="cuda")
    buf[..., :width] = t.to(DT[dt])
    return buf[..., :width]


def _rows_8bit(g, rows, width, scale=1.0, lead=()):
    """Normal values as e4m3 codes and one scale a row."""
    t = torch.randn((*lead, rows, width), generator=g, device="cuda") * scale
    s = t.abs().amax(-1) / 448.0
    buf = torch.zeros((*lead, rows, _ld(width, "e4m3")), dtype=torch.uint8, device="cuda")
    buf[..., :width] = (t / s[..., None]).to(DT["e4m3"]).view(torch.uint8)
    return buf.view(DT["e4m3"])[..., :width], s


def _ids(g, n, rows):
    """Skewed ids: rank r drawn about as r^-1, spread over the table by a fixed stride."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = ((rows + 1.0) ** u - 1.0).long().clamp_(0, rows - 1)
    return ((rank * 7919 + 13) % rows).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "lookup":
        s["table"] = (torch.randn((case["rows"], case["d"]), generator=g, device="cuda") * case["d"] ** -0.5).to(DT[case["table"]])
        s["ids"] = _ids(g, case["n"], case["rows"])
        s["scale"] = math.sqrt(case["d"])
        s["out"] = torch.empty((case["n"], case["d"]), dtype=DT[case["out"]], device="cuda")
    elif op == "lookup_grad":
        s["ids"] = _ids(g, case["n"], case["rows"])
        s["dout"] = torch.randn((case["n"], case["d"]), generator=g, device="cuda").to(DT[case["grad"]])
        s["scale"] = math.sqrt(case["d"])
        s["dtable"] = torch.empty((case["rows"], case["d"]), dtype=DT[case["table"]], device="cuda")
    elif op == "norm":
        rows, d, x = case["rows"], case["d"], DT[case["x"]]
        s["x"] = torch.randn((rows, d), generator=g, device="cuda").to(x)
        s["residual"] = (torch.randn((rows, d), generator=g, device="cuda") * 2).to(x) if case["residual"] else None
        s["w"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        s["eps"] = 1e-6
        s["y"] = torch.empty((rows, d), dtype=DT[case["y"]], device="cuda")
        s["h"] = torch.empty((rows, d), dtype=x, device="cuda") if case["residual"] else None
        s["rstd"] = torch.empty(rows, device="cuda")
        s["y_scale"] = torch.empty(rows, device="cuda") if case["y"] == "e4m3" else None
    elif op == "norm_grad":
        rows, d, x = case["rows"], case["d"], DT[case["x"]]
        s["h"] = (torch.randn((rows, d), generator=g, device="cuda") * 2).to(x)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + 1e-6).float()
        s["w"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        s["dy"] = torch.randn((rows, d), generator=g, device="cuda").to(x)
        s["dh"] = torch.randn((rows, d), generator=g, device="cuda").to(x) if case["residual"] else None
        s["dx"] = torch.empty((rows, d), dtype=x, device="cuda")
        s["dw"] = torch.empty(d, device="cuda")
    elif op == "dropout":
        x = DT[case["x"]]
        s["x"] = torch.randn(case["n"], generator=g, device="cuda").to(x)
        s["residual"] = torch.randn(case["n"], generator=g, device="cuda").to(x) if case["residual"] else None
        s["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda")
        s["y"] = torch.empty(case["n"], dtype=x, device="cuda")
    else:
        M, spare, E, N, K = (case[k] for k in ("M", "spare", "E", "N", "K"))
        # routed rows per expert: a router's uneven shares, now and then none
        share = torch.rand(E, generator=g, device="cuda").square() + 0.05
        pick = torch.multinomial(share, M, replacement=True, generator=g)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = torch.bincount(pick, minlength=E).cumsum(0).to(torch.int32)
        s["most"] = int(torch.bincount(pick, minlength=E).max())      # the longest expert's rows
        if case["x"] == "e4m3":
            s["X"], s["x_scale"] = _rows_8bit(g, M + spare, K)
            s["W"], s["w_scale"] = _rows_8bit(g, N, K, K ** -0.5, (E,))
        else:
            s["X"], s["x_scale"] = _rows(g, M + spare, K, case["x"]), None
            s["W"], s["w_scale"] = _rows(g, N, K, case["x"], K ** -0.5, (E,)), None
        if op == "experts":
            s["bias"] = 0.1 * torch.randn((E, N), generator=g, device="cuda")
            s["Y"] = torch.zeros((M + spare, _ld(N, case["y"])), dtype=DT[case["y"]], device="cuda")[:, :N]
        else:
            s["dY"] = _rows(g, M + spare, N, case["x"])
            # the forward's outputs: what ReLU left, for a half of the places nothing
            s["Y"] = _rows(g, M + spare, N, case["x"]).clamp_(min=0) if case["relu"] else None
            s["dX"] = torch.zeros((M + spare, _ld(K, case["x"])), dtype=DT[case["x"]], device="cuda")[:, :K]
            s["dW"] = torch.zeros((E, N, _ld(K, case["dw"])), dtype=DT[case["dw"]], device="cuda")[..., :K]
            s["db"] = torch.empty((E, N), device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def _own_pass(s):
    import embedding_bags_dot_b200 as E

    c = s["case"]
    op = c["op"]
    act = E.ACT_RELU if c.get("relu") else E.ACT_NONE
    if "ws" not in s:   # a user's program keeps its workspace and table handle from call to call
        need = E.ERR_RECORD_BYTES
        if op == "lookup":
            s["T"] = E.Tables(s["table"], [c["rows"]], c["d"])
        elif op == "lookup_grad":
            need = E.dlrm_embed_bwd_workspace_size(c["rows"], c["d"], c["n"])
        elif op == "norm_grad":
            need = E.dlrm_rmsnorm_bwd_workspace_size(c["rows"], c["d"])
        elif op == "experts_grad":
            need = E.dlrm_experts_bwd_workspace_size(c["E"], c["M"] + c["spare"], c["N"], c["K"], act)
        s["ws"] = E.alloc_workspace(need)
    if op == "lookup":
        E.dlrm_embed_fwd(s["T"], 0, s["ids"], s["out"], s["ws"], scale=s["scale"])
        return s["out"]
    if op == "lookup_grad":
        E.dlrm_embed_bwd(s["ids"], s["dout"], s["dtable"], s["ws"], scale=s["scale"])
        return s["dtable"]
    if op == "norm":
        E.dlrm_rmsnorm_fwd(s["x"], s["w"], s["y"], eps=s["eps"], residual=s["residual"], h=s["h"],
                           y_scale=s["y_scale"], rstd=s["rstd"])
        return {"y": s["y"], "y_scale": s["y_scale"], "h": s["h"], "rstd": s["rstd"]}
    if op == "norm_grad":
        E.dlrm_rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["w"], s["dx"], s["ws"], dw=s["dw"], dh=s["dh"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "dropout":
        E.dlrm_dropout(s["x"], s["y"], c["p"], s["rng"], residual=s["residual"])
        return s["y"]
    if op == "experts":
        E.dlrm_experts_fwd(s["X"], s["W"], s["offsets"], s["Y"], s["ws"], bias=s["bias"], act=act,
                           x_scale=s["x_scale"], w_scale=s["w_scale"])
        return s["Y"]
    E.dlrm_experts_bwd(s["dY"], s["X"], s["W"], s["offsets"], s["ws"], Y=s["Y"], act=act, dX=s["dX"], dW=s["dW"],
                       db=s["db"])
    return {"dX": s["dX"], "dW": s["dW"], "db": s["db"]}


def _philox_words(n4, rng):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
    words 0..3 of counters 0..n4-1, key = rng[0], upper counter half = rng[1], as int64 [n4][4]."""
    low = 0xFFFFFFFF
    i = torch.arange(n4, dtype=torch.int64, device=rng.device)
    c0, c1 = i & low, i >> 32
    c2, c3 = (rng[1] & low).expand(n4), ((rng[1] >> 32) & low).expand(n4)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57       # modulo 2^64
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), 1)


def _padded(s):
    """Row numbers [E][most] of each expert's rows, which of them are real, and each row's place in that."""
    offs = s["offsets"].long()
    at = offs[:-1, None] + torch.arange(s["most"], device=offs.device)
    real = at < offs[1:, None]
    rows = s["X"].shape[0]
    r = torch.arange(rows, device=offs.device)
    e = torch.searchsorted(offs[1:].contiguous(), r, right=True)
    inside = (r < offs[-1]) & (r >= offs[0])
    e = torch.where(inside, e, torch.zeros_like(e))
    place = torch.where(inside, e * s["most"] + r - offs[e], torch.zeros_like(r))
    return at.clamp(max=rows - 1), real[..., None], place, inside[:, None]


def _values(q, scale):
    return q.float() if scale is None else q.float() * scale[..., None]


def run(s):
    if own:
        return _own_pass(s)
    c = s["case"]
    op = c["op"]
    if op == "lookup":
        return (s["table"][s["ids"].long()].float() * s["scale"]).to(DT[c["out"]])
    if op == "lookup_grad":
        total = torch.zeros((c["rows"], c["d"]), device="cuda").index_add_(0, s["ids"].long(), s["dout"].float())
        return (total * s["scale"]).to(DT[c["table"]])
    if op == "norm":
        h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
        rstd = 1 / torch.sqrt((h * h).mean(1) + s["eps"])
        y = h * rstd[:, None] * s["w"]
        scale = None
        if c["y"] == "e4m3":
            scale = y.abs().amax(1) / 448.0
            y = y / scale[:, None]
        return {"y": y.to(DT[c["y"]]), "y_scale": scale, "h": None if s["residual"] is None else h.to(DT[c["x"]]),
                "rstd": rstd}
    if op == "norm_grad":
        xh = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        u = dy * s["w"]
        dx = s["rstd"][:, None] * (u - xh * (u * xh).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(DT[c["x"]]), "dw": (dy * xh).sum(0)}
    if op == "dropout":
        n = c["n"]
        words = _philox_words((n + 3) // 4, s["rng"]).reshape(-1)[:n]
        kept = words >= round(c["p"] * 2 ** 32)
        y = torch.where(kept, s["x"].float() * (1 / (1 - c["p"])), 0.0)
        return (y if s["residual"] is None else y + s["residual"].float()).to(DT[c["x"]])
    at, real, place, inside = _padded(s)
    W = _values(s["W"], s["w_scale"])
    if op == "experts":
        x = _values(s["X"], s["x_scale"])[at]
        y = torch.bmm(x, W.transpose(1, 2)) + s["bias"][:, None]
        if c["relu"]:
            y = torch.clamp(y, min=0)
        y = y.reshape(-1, c["N"])[place].to(DT[c["y"]])
        return torch.where(inside, y, s["Y"])
    dp = s["dY"].float()
    if c["relu"]:
        dp = torch.where(s["Y"] > 0, dp, 0.0)
    dp = torch.where(real, dp[at], 0.0)
    x = torch.where(real, s["X"].float()[at], 0.0)
    dx = torch.bmm(dp, W).reshape(-1, c["K"])[place].to(DT[c["x"]])
    return {"dX": torch.where(inside, dx, s["dX"]), "dW": torch.bmm(dp.transpose(1, 2), x).to(DT[c["dw"]]),
            "db": dp.sum(1)}


# ------------------------------------------------------------------ the least of a pass

def work(c):
    op = c["op"]
    if op == "lookup":
        return {"bytes": c["n"] * (4 + c["d"] * (SIZE[c["table"]] + SIZE[c["out"]])), "flops": c["n"] * c["d"]}
    if op == "lookup_grad":
        return {"bytes": c["n"] * (4 + c["d"] * SIZE[c["grad"]]) + c["rows"] * c["d"] * SIZE[c["table"]],
                "flops": 2 * c["n"] * c["d"]}
    if op == "norm":
        x, y = SIZE[c["x"]], SIZE[c["y"]]
        row = c["d"] * (x + y + (2 * x if c["residual"] else 0)) + 4 + (4 if c["y"] == "e4m3" else 0)
        return {"bytes": c["rows"] * row + 4 * c["d"], "flops": 6 * c["rows"] * c["d"]}
    if op == "norm_grad":
        row = c["d"] * SIZE[c["x"]] * (4 if c["residual"] else 3) + 4
        return {"bytes": c["rows"] * row + 8 * c["d"], "flops": 10 * c["rows"] * c["d"]}
    if op == "dropout":
        return {"bytes": c["n"] * SIZE[c["x"]] * (3 if c["residual"] else 2) + 16, "flops": 3 * c["n"]}
    M, E, N, K, x = c["M"], c["E"], c["N"], c["K"], SIZE[c["x"]]
    used = min(E, M)     # experts that can have rows
    if op == "experts":
        scales = 4 * (M + used * N) if c["x"] == "e4m3" else 0
        return {"bytes": M * K * x + used * N * (K * x + 4) + M * N * SIZE[c["y"]] + scales, "flops": 2 * M * N * K}
    return {"bytes": M * N * x * (2 if c["relu"] else 1) + 2 * M * K * x + used * N * K * x
            + E * N * (K * SIZE[c["dw"]] + 4), "flops": 4 * M * N * K}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _philox_numpy(n4, key, upper):
    """The generator's words by numpy's unsigned 64-bit products, [n4][4] uint32."""
    c = np.zeros((4, n4), dtype=np.uint64)
    c[0] = np.arange(n4, dtype=np.uint64)
    c[2], c[3] = upper & 0xFFFFFFFF, upper >> 32
    k = [key & 0xFFFFFFFF, key >> 32]
    m32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for r in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        n0 = (p1 >> sh) ^ c[1] ^ np.uint64((k[0] + r * 0x9E3779B9) % 2 ** 32)
        n2 = (p0 >> sh) ^ c[3] ^ np.uint64((k[1] + r * 0xBB67AE85) % 2 ** 32)
        c[0], c[1], c[2], c[3] = n0, p1 & m32, n2, p0 & m32
    return c.T.astype(np.uint32)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "lookup":
        rows = torch.index_select(s["table"], 0, s["ids"])
        return rows.double().mul_(s["scale"])
    if op == "lookup_grad":
        ids, order = torch.sort(s["ids"].long(), stable=True)
        # running sums within each run of equal ids, taken as differences would lose bits: add row by row instead
        out = torch.zeros((c["rows"], c["d"]), dtype=torch.float64, device="cuda")
        return out.index_put_((ids,), s["dout"][order].double() * s["scale"], accumulate=True)
    if op == "norm":
        t = s["x"].double()
        if s["residual"] is not None:
            t = t.add_(s["residual"].double())
        inv = (t.pow(2).sum(1) / c["d"] + s["eps"]).pow(-0.5)
        y = torch.einsum("rd,r,d->rd", t, inv, s["w"].double())
        scale = None
        if c["y"] == "e4m3":
            scale = torch.maximum(y.amax(1), -y.amin(1)) / 448
            y = y / scale.unsqueeze(1)
        return {"y": y, "y_scale": scale, "h": None if s["residual"] is None else t, "rstd": inv}
    if op == "norm_grad":
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double().unsqueeze(1)
        along = torch.einsum("rd,rd,d->r", h, dy, w).unsqueeze(1)
        dx = r * dy * w - h * r.pow(3) * along / c["d"]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("rd,rd,r->d", dy, h, r.squeeze(1))}
    if op == "dropout":
        key, upper = (int(v) for v in s["rng"].tolist())
        word = torch.from_numpy(_philox_numpy((c["n"] + 3) // 4, key, upper).reshape(-1)[:c["n"]].astype(np.int64)).cuda()
        y = s["x"].double() / (1 - c["p"])
        y[word < round(c["p"] * 2 ** 32)] = 0
        return y if s["residual"] is None else y + s["residual"].double()
    ends = s["offsets"].tolist()
    X, W = s["X"].double(), s["W"]
    if s["x_scale"] is not None:
        X = X * s["x_scale"].double().unsqueeze(1)
    if op == "experts":
        Y = s["Y"].double()
        for e in range(c["E"]):
            a, b = ends[e], ends[e + 1]
            We = W[e].double() if s["w_scale"] is None else W[e].double() * s["w_scale"][e].double().unsqueeze(1)
            y = X[a:b] @ We.T + s["bias"][e].double()
            Y[a:b] = y.relu() if c["relu"] else y
        return Y
    dX, dW = s["dX"].double(), torch.zeros((c["E"], c["N"], c["K"]), dtype=torch.float64, device="cuda")
    db = torch.zeros((c["E"], c["N"]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        a, b = ends[e], ends[e + 1]
        dp = s["dY"][a:b].double()
        if c["relu"]:
            dp = dp * (s["Y"][a:b] > 0)
        dX[a:b] = dp @ W[e].double()
        dW[e] = dp.T @ X[a:b]
        db[e] = dp.sum(0)
    return {"dX": dX, "dW": dW, "db": db}
