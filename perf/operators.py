"""Cases and plain forms of the operators around the FP8 GEMMs of a mixture-of-experts block:

  norm_residual            post-norm of a block's output, gate, residual scale, residual sum, and the
                           next block's pre-norm (bf16 / f32 rows, or FP8 codes and 1x128 scales)
  norm_residual_backward   its gradients: residual stream, block output, both norms' weights, gate
  moe_permute              tokens sorted by expert into the contiguous layout, not quantised
  moe_permute_backward     its gradient: the rows of a token's slots summed
  moe_combine_backward     gradient of the weighted combine: rows (bf16, or FP8 codes and 1x128
                           scales for the next grouped GEMM) and routing weights
  moe_dispatch_masked      tokens quantised into the masked (decode) layout

`run` takes what `prepare` gives and makes one pass, in the plain form below or, with `own` set,
through the library.  Buffers whose unused rows an operator leaves as they were (unused blocks, rows
behind masked_m, the tail of a scale row) are the state's own and start at zero.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def norm_case(name, rows, H, dtype, post, gate, res, quant, backward):
    return dict(name=name, op="norm_backward" if backward else "norm", rows=rows, H=H, dtype=dtype, post=post,
                gate=gate, res=res, quant=quant)


def moe_case(name, op, T, topk, G, N, dtype, drop, quant=False, Mmax=0):
    return dict(name=name, op=op, T=T, topk=topk, G=G, N=N, dtype=dtype, drop=drop, quant=quant, Mmax=Mmax)


def listed():
    return [
        # one decoded token between two blocks: post-norm, residual, pre-norm, quantised for the next GEMM
        norm_case("norm_token_fp8", 1, 7168, "bf16", True, "none", True, True, False),
        # a prefill / training batch with a per-channel gate, bf16 rows out (for a router and a dispatch)
        norm_case("norm_batch_bf16", 8192, 7168, "bf16", True, "channel", True, False, False),
        # the same batch's backward pass
        norm_case("norm_backward_bf16", 8192, 7168, "bf16", True, "channel", True, False, True),
        # FP32 training of a narrow model on a ragged batch, with a gate per token
        norm_case("norm_backward_f32", 1021, 2112, "f32", True, "token", True, False, True),
        # a training batch's tokens sorted by expert
        moe_case("permute_bf16", "permute", 4096, 8, 64, 7168, "bf16", 0.0),
        # a small ragged FP32 batch with dropped slots
        moe_case("permute_f32", "permute", 333, 3, 7, 2112, "f32", 0.2),
        # gradients of the sorted rows back to the tokens
        moe_case("permute_backward_bf16", "permute_backward", 4096, 8, 64, 7168, "bf16", 0.0),
        moe_case("permute_backward_f32", "permute_backward", 129, 3, 7, 520, "f32", 0.2),
        # gradient of the combine, quantised for the FP8 grouped GEMM that follows it
        moe_case("combine_backward_fp8", "combine_backward", 4096, 8, 64, 7168, "bf16", 0.0, quant=True),
        # the same in bf16 on a small ragged batch with dropped slots
        moe_case("combine_backward_bf16", "combine_backward", 333, 4, 16, 4096, "bf16", 0.1),
        # one decoded token sent to its experts
        moe_case("dispatch_masked_token", "dispatch_masked", 1, 8, 16, 7168, "bf16", 0.0, Mmax=256),
        # a full decode batch: up to 256 rows per expert
        moe_case("dispatch_masked_batch", "dispatch_masked", 256, 8, 16, 7168, "bf16", 0.0, Mmax=256),
    ]


def log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    """Rows from one token to a large batch, widths from 64 to 16384 (multiples of a 16-byte vector, of
    128 where codes are quantised), every type, gate and direction."""
    limit = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["norm", "norm_backward", "permute", "permute_backward", "combine_backward",
                         "dispatch_masked"])
        if op.startswith("norm"):
            quant = op == "norm" and rng.random() < 0.5
            c = norm_case("", log_int(rng, 1, 32768), log_int(rng, 128, 16384, 128 if quant else 8),
                          rng.choice(["bf16", "f32"]), rng.random() < 0.75, rng.choice(["none", "channel", "token"]),
                          rng.random() < 0.8, quant, op == "norm_backward")
        else:
            G = log_int(rng, 2, 256)
            topk = rng.randint(1, min(16, G))
            quant = op == "combine_backward" and rng.random() < 0.5
            fp8 = quant or op == "dispatch_masked"
            N = log_int(rng, 128, 8192, 128) if fp8 else log_int(rng, 64, 8192, 8)
            dtype = "bf16" if op == "combine_backward" else rng.choice(["bf16", "f32"])
            if op == "dispatch_masked":
                T = log_int(rng, 1, 1024)
                # room for every token at one expert, or a tighter capacity that may overflow
                Mmax = rng.choice([(T + 127) // 128 * 128, 4 * ((2 * T * topk // G + 4) // 4)])
            else:
                T, Mmax = log_int(rng, 1, 16384), 0
            c = moe_case("", op, T, topk, G, N, dtype, rng.choice([0.0, 0.05, 0.3]), quant, Mmax)
            # the masked buffers, most of them unused, stay small next to the card
            if op == "dispatch_masked" and G * Mmax * N > 1 << 30:
                continue
        if work(c)["bytes"] <= limit:
            del c["name"]
            return c


def work(case):
    """Bytes: every input read once, every output written once (routed rows at their expected number;
    padding rows not counted).  Flops: about what the formulas need."""
    c = case
    if c["op"].startswith("norm"):
        n, e = c["rows"] * c["H"], 2 if c["dtype"] == "bf16" else 4
        vecs = 1 + c["post"] + (c["gate"] == "channel")
        small = 4 * c["H"] * vecs + (4 * c["rows"] if c["gate"] == "token" else 0)
        if c["op"] == "norm":
            out = n * e + (n + n // 32 if c["quant"] else n * e)
            return {"bytes": n * e * (1 + c["res"]) + out + small, "flops": 12.0 * n}
        # reads dz, dh_out, h_out, y; writes dh, dy and the small gradients
        return {"bytes": n * e * 6 + 2 * small, "flops": 30.0 * n}
    R = c["T"] * c["topk"]
    live, e, N = R * (1.0 - c["drop"]), 2 if c["dtype"] == "bf16" else 4, c["N"]
    if c["op"] == "permute":
        return {"bytes": c["T"] * N * e + live * N * e + 8 * R, "flops": 0.0}
    if c["op"] == "permute_backward":
        return {"bytes": live * N * e + c["T"] * N * e + 4 * R, "flops": live * N}
    if c["op"] == "combine_backward":
        out = N + N / 32 if c["quant"] else 2 * N
        return {"bytes": c["T"] * N * 2 + live * (2 * N + out) + 12 * R, "flops": (8.0 if c["quant"] else 3.0) * live * N}
    return {"bytes": c["T"] * N * e + live * (N + N / 32) + 8 * R, "flops": 4.0 * c["T"] * N}


# ---------------------------------------------------------------- inputs
def blocks_of(c):
    return (c["T"] * c["topk"] + 127) // 128 + c["G"]


def routing(c, gen):
    """A router's output: top-k of logits with popular and unpopular experts, softmax weights, and a
    share of dropped slots (-1)."""
    T, topk, G = c["T"], c["topk"], c["G"]
    logits = torch.randn(T, G, device=DEVICE, generator=gen) + 0.5 * torch.randn(G, device=DEVICE, generator=gen)
    best = torch.topk(logits, topk, dim=1)
    w = torch.softmax(best.values, dim=1).reshape(-1).contiguous()
    expert = best.indices.to(torch.int32).reshape(-1)
    if c["drop"]:
        gone = torch.rand(expert.shape, device=DEVICE, generator=gen) < c["drop"]
        expert = torch.where(gone, torch.full_like(expert, -1), expert)
    return expert.contiguous(), w


def activations(rows, width, dtype, gen, scale=1.0):
    """N(0, scale) with one channel in 64 ten times as large, as residual streams have."""
    x = torch.randn(rows, width, device=DEVICE, generator=gen) * scale
    x[:, ::64] *= 10.0
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = {"c": c}
    if c["op"].startswith("norm"):
        rows, H, dt = c["rows"], c["H"], c["dtype"]
        s["y"] = activations(rows, H, dt, gen, 0.5)
        s["post_w"] = 1.0 + 0.2 * torch.randn(H, device=DEVICE, generator=gen) if c["post"] else None
        s["pre_w"] = 1.0 + 0.2 * torch.randn(H, device=DEVICE, generator=gen)
        shape = {"none": None, "channel": (H,), "token": (rows, 1)}[c["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(torch.randn(shape, device=DEVICE, generator=gen))
        s["scale"] = 0.5
        h = activations(rows, H, dt, gen)
        if c["op"] == "norm":
            s["h"] = h if c["res"] else None
            ld = max(4, (rows + 3) // 4 * 4)
            s["out"] = None
            if c["quant"]:
                s["out"] = (torch.empty_like(h), torch.empty(rows, H, dtype=torch.uint8, device=DEVICE),
                            torch.zeros(H // 128, ld, device=DEVICE))
        else:
            s["h_out"] = h
            s["dz"] = torch.randn(rows, H, device=DEVICE, generator=gen).to(DTYPES[dt])
            s["dh_out"] = torch.randn(rows, H, device=DEVICE, generator=gen).to(DTYPES[dt])
        return s
    T, topk, G, N, dt = c["T"], c["topk"], c["G"], c["N"], DTYPES[c["dtype"]]
    R, M = T * topk, blocks_of(c) * 128
    expert, w = routing(c, gen)
    if c["op"] == "permute":
        s["x"] = activations(T, N, c["dtype"], gen)
        s["expert"] = expert
        s["out"] = (torch.zeros(M, N, dtype=dt, device=DEVICE), torch.empty(R, dtype=torch.int32, device=DEVICE),
                    torch.empty(M // 128, dtype=torch.int32, device=DEVICE))
    elif c["op"] == "permute_backward":
        s["pos"] = contiguous_layout(expert, G, M // 128)[0]
        s["dxs"] = torch.randn(M, N, device=DEVICE, generator=gen).to(dt)
    elif c["op"] == "combine_backward":
        s["pos"] = contiguous_layout(expert, G, M // 128)[0]
        s["w"] = w
        s["dout"] = torch.randn(T, N, device=DEVICE, generator=gen).to(dt)
        s["D"] = activations(M, N, c["dtype"], gen)
        dw = torch.empty(R, device=DEVICE)
        if c["quant"]:
            s["out"] = (torch.zeros(M, N, dtype=torch.uint8, device=DEVICE), torch.zeros(N // 128, M, device=DEVICE), dw)
        else:
            s["out"] = (torch.zeros(M, N, dtype=dt, device=DEVICE), dw)
    else:
        s["x"] = activations(T, N, c["dtype"], gen)
        s["expert"] = expert
        s["out"] = (torch.zeros(G, c["Mmax"], N, dtype=torch.uint8, device=DEVICE),
                    torch.zeros(G, N // 128, c["Mmax"], device=DEVICE),
                    torch.empty(R, dtype=torch.int32, device=DEVICE),
                    torch.empty(G, dtype=torch.int32, device=DEVICE))
    return s


# ---------------------------------------------------------------- the plain forms
def expert_ranks(expert, G):
    """(key, rank, counts): each slot's expert (G where dropped), its rank among the earlier slots of
    that expert, and the slots of each expert."""
    key = torch.where(expert < 0, G, expert).long()
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(G + 1, dtype=torch.int64, device=key.device).scatter_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(counts, 0) - counts
    ranks = torch.empty_like(key)
    ranks[order] = torch.arange(key.numel(), device=key.device) - first[key[order]]
    return key, ranks, counts[:G]


def contiguous_layout(expert, G, blocks):
    """pos and m_indices of the contiguous layout: segments in expert order, padded to 128 rows."""
    key, ranks, counts = expert_ranks(expert, G)
    ends = torch.cumsum((counts + 127) // 128, 0)
    off = torch.cat([(ends - (counts + 127) // 128) * 128, ends.new_zeros(1)])
    pos = torch.where(key < G, off[key] + ranks, -1).to(torch.int32)
    b = torch.arange(blocks, device=key.device)
    m = torch.searchsorted(ends, b, right=True)
    return pos, torch.where(b < ends[-1], m, -1).to(torch.int32)


def slot_of_row(pos, M):
    """For each row of the layout the slot that fills it, -1 where none does."""
    inv = torch.full((M + 1,), -1, dtype=torch.int64, device=pos.device)
    inv[torch.where(pos < 0, M, pos.long())] = torch.arange(pos.numel(), device=pos.device)
    return inv[:M]


def quantised(v):
    """FP32 rows -> e4m3 values and scales [rows, groups], per 1x128 group."""
    g = v.view(v.shape[0], -1, 128)
    amax = g.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (g / scale[..., None]).clamp(-448.0, 448.0).to(FP8).view(v.shape), scale


def plain_norm(s):
    c, y = s["c"], s["y"].float()
    p = y
    if c["post"]:
        p = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["post_w"]
    if s["gate"] is not None:
        p = p * s["gate"]
    h = p * s["scale"]
    if s["h"] is not None:
        h = h + s["h"].float()
    z = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["pre_w"]
    dt = s["y"].dtype
    if not c["quant"]:
        return h.to(dt), z.to(dt)
    q, sc = quantised(z)
    sa = torch.zeros_like(s["out"][2])
    sa[:, : c["rows"]] = sc.T
    return h.to(dt), q, sa


def plain_norm_backward(s):
    c, dt = s["c"], s["y"].dtype
    h, y, dz = s["h_out"].float(), s["y"].float(), s["dz"].float()
    r1 = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n1 = h * r1
    dn = dz * s["pre_w"]
    dpre = (dz * n1).sum(0)
    dh = s["dh_out"].float() + r1 * (dn - n1 * (dn * n1).mean(-1, keepdim=True))
    g = 1.0 if s["gate"] is None else s["gate"]
    if c["post"]:
        r2 = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        u = y * r2
        dp = s["scale"] * g * dh
        dpost = (dp * u).sum(0)
        du = dp * s["post_w"]
        dy = r2 * (du - u * (du * u).mean(-1, keepdim=True))
        p = u * s["post_w"]
    else:
        dpost, dy, p = None, s["scale"] * g * dh, y
    dg = None
    if c["gate"] == "channel":
        dg = (s["scale"] * p * dh).sum(0)
    elif c["gate"] == "token":
        dg = (s["scale"] * p * dh).sum(-1, keepdim=True)
    return dh.to(dt), dy.to(dt), dpre, dpost, dg


def plain_permute(s):
    c = s["c"]
    xs, _, mi = s["out"]
    pos, m_indices = contiguous_layout(s["expert"], c["G"], mi.numel())
    inv = slot_of_row(pos, xs.shape[0])
    rows = s["x"][(inv.clamp(min=0) // c["topk"])]
    return torch.where((inv >= 0)[:, None], rows, torch.zeros_like(rows)), pos, m_indices


def plain_permute_backward(s):
    c, pos = s["c"], s["pos"].long()
    rows = s["dxs"][pos.clamp(min=0)].float() * (pos >= 0)[:, None]
    return rows.view(c["T"], c["topk"], -1).sum(1).to(s["dxs"].dtype)


def plain_combine_backward(s):
    c, pos = s["c"], s["pos"].long()
    dout = s["dout"].float()
    rows = s["D"][pos.clamp(min=0)].float().view(c["T"], c["topk"], -1)
    dw = (rows * dout[:, None, :]).sum(-1).view(-1) * (pos >= 0)
    inv = slot_of_row(s["pos"], s["D"].shape[0])
    live, slot = inv >= 0, inv.clamp(min=0)
    v = dout[slot // c["topk"]] * (s["w"][slot] * live)[:, None]
    if not c["quant"]:
        return v.to(s["D"].dtype), dw
    q, sc = quantised(v)
    return q, (sc * live[:, None]).T.contiguous(), dw


def plain_dispatch_masked(s):
    c = s["c"]
    G, Mmax, K = s["out"][0].shape
    key, ranks, counts = expert_ranks(s["expert"], G)
    pos = torch.where((key < G) & (ranks < Mmax), key * Mmax + ranks, -1).to(torch.int32)
    inv = slot_of_row(pos, G * Mmax)
    live, tok = inv >= 0, inv.clamp(min=0) // c["topk"]
    q, sc = quantised(s["x"].float())
    A = torch.where(live[:, None], q.view(torch.uint8)[tok], 0).to(torch.uint8).view(G, Mmax, K)
    sa = (sc[tok] * live[:, None]).view(G, Mmax, -1).transpose(1, 2).contiguous()
    return A.view(FP8), sa, pos, counts.clamp(max=Mmax).to(torch.int32)


PLAIN = {"norm": plain_norm, "norm_backward": plain_norm_backward, "permute": plain_permute,
         "permute_backward": plain_permute_backward, "combine_backward": plain_combine_backward,
         "dispatch_masked": plain_dispatch_masked}


def run(state):
    s, c = state, state["c"]
    if not own:
        return PLAIN[c["op"]](s)
    from fp8_block_scaled_x128_b200 import gemm
    op = c["op"]
    if op == "norm":
        r = gemm.norm_residual(s["y"], s["h"], post_weight=s["post_w"], gate=s["gate"], scale=s["scale"],
                               pre_weight=s["pre_w"], eps=EPS, quantize=c["quant"], out=s["out"])
        return (r[0], r[1].view(FP8), r[2]) if c["quant"] else r
    if op == "norm_backward":
        return gemm.norm_residual_backward(s["dz"], s["dh_out"], s["h_out"], s["y"], post_weight=s["post_w"],
                                           gate=s["gate"], scale=s["scale"], pre_weight=s["pre_w"], eps=EPS)
    if op == "permute":
        return gemm.moe_permute(s["x"], s["expert"], c["topk"], c["G"], out=s["out"])
    if op == "permute_backward":
        return gemm.moe_permute_backward(s["dxs"], s["pos"], c["T"], c["topk"])
    if op == "combine_backward":
        r = gemm.moe_combine_backward(s["dout"], s["D"], s["pos"], s["w"], c["T"], c["topk"], quantize=c["quant"],
                                      out=s["out"])
        return (r[0].view(FP8), r[1], r[2]) if c["quant"] else r
    A, sa, pos, masked_m = gemm.moe_dispatch_masked(s["x"], s["expert"], c["topk"], c["G"], c["Mmax"], out=s["out"])
    return A.view(FP8), sa, pos, masked_m


# ---------------------------------------------------------------- the definitions in 64 bits
def exact_codes(v):
    """Unrounded quotients and scales of 1x128 groups, in 64 bits."""
    rows, K = v.shape
    q, scale = torch.empty_like(v), v.new_empty(rows, K // 128)
    for kb in range(K // 128):
        part = v[:, 128 * kb:128 * kb + 128]
        a = part.abs().max(dim=1).values
        scale[:, kb] = torch.where(a == 0, torch.ones_like(a), a / 448)
        q[:, 128 * kb:128 * kb + 128] = part / scale[:, kb:kb + 1]
    return q, scale


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "norm":
        H = c["H"]
        b = s["y"].double() * s["scale"]
        if c["post"]:
            b = b * s["post_w"].double() / torch.sqrt((s["y"].double() ** 2).sum(1, keepdim=True) / H + EPS)
        if c["gate"] != "none":
            b = b * s["gate"].double()
        h = b if s["h"] is None else s["h"].double() + b
        z = h * s["pre_w"].double() / torch.sqrt((h ** 2).sum(1, keepdim=True) / H + EPS)
        if not c["quant"]:
            return h, z
        q, sc = exact_codes(z)
        sa = torch.zeros(s["out"][2].shape, dtype=torch.float64, device=DEVICE)
        sa[:, :c["rows"]] = sc.T
        return h, q, sa
    if c["op"] == "norm_backward":
        # d/dx of x w / sqrt(mean(x^2) + eps): w g / d - x <x, w g> / (H d^3)
        H = c["H"]
        h, y, dz = s["h_out"].double(), s["y"].double(), s["dz"].double()
        d = torch.sqrt((h ** 2).sum(1, keepdim=True) / H + EPS)
        wg = dz * s["pre_w"].double()
        dh = s["dh_out"].double() + wg / d - h * (h * wg).sum(1, keepdim=True) / (H * d ** 3)
        dpre = (dz * h / d).sum(0)
        gate = torch.ones(1, 1, dtype=torch.float64, device=DEVICE) if s["gate"] is None else s["gate"].double()
        b = s["scale"] * dh          # gradient of gate * N(y)
        dpost = None
        if c["post"]:
            w = s["post_w"].double()
            e = torch.sqrt((y ** 2).sum(1, keepdim=True) / H + EPS)
            dg = b * w * y / e
            dpost = (b * gate * y / e).sum(0)
            wg = b * gate * w
            dy = wg / e - y * (y * wg).sum(1, keepdim=True) / (H * e ** 3)
        else:
            dg, dy = b * y, b * gate
        dg = {"none": None, "channel": dg.sum(0), "token": dg.sum(1, keepdim=True)}[c["gate"]]
        return dh, dy, dpre, dpost, dg
    T, topk, G, N = c["T"], c["topk"], c["G"], c["N"]
    token = torch.arange(T * topk, device=DEVICE) // topk
    if c["op"] in ("permute", "dispatch_masked"):
        # walk the experts: each takes its slots in order
        slots = [torch.nonzero(s["expert"] == g).view(-1) for g in range(G)]
    if c["op"] == "permute":
        xs = torch.zeros(s["out"][0].shape, dtype=torch.float64, device=DEVICE)
        at = 0
        for sl in slots:
            xs[at:at + sl.numel()] = s["x"][token[sl]].double()
            at += (sl.numel() + 127) // 128 * 128
        return xs, None, None
    if c["op"] == "dispatch_masked":
        q, sc = exact_codes(s["x"].double())
        A = torch.zeros(s["out"][0].shape, dtype=torch.float64, device=DEVICE)
        sa = torch.zeros(s["out"][1].shape, dtype=torch.float64, device=DEVICE)
        for g, sl in enumerate(slots):
            sl = sl[:c["Mmax"]]
            A[g, :sl.numel()] = q[token[sl]]
            sa[g, :, :sl.numel()] = sc[token[sl]].T
        return A, sa, None, None
    live = torch.nonzero(s["pos"] >= 0).view(-1)
    row = s["pos"][live].long()
    if c["op"] == "permute_backward":
        dx = torch.zeros(T, N, dtype=torch.float64, device=DEVICE)
        for k in range(topk):
            mine = live % topk == k
            dx[token[live[mine]]] += s["dxs"][row[mine]].double()
        return dx
    dD = torch.zeros(s["D"].shape, dtype=torch.float64, device=DEVICE)
    dw = torch.zeros(T * topk, dtype=torch.float64, device=DEVICE)
    for part in torch.arange(live.numel(), device=DEVICE).split(4096):
        r, sl = row[part], live[part]
        g = s["dout"][token[sl]].double()
        dw[sl] = (g * s["D"][r].double()).sum(1)
        dD[r] = g * s["w"][sl].double()[:, None]
    if not c["quant"]:
        return dD, dw
    q, sc = exact_codes(dD[row])
    dD[row] = q
    sa = torch.zeros(s["out"][1].shape, dtype=torch.float64, device=DEVICE)
    sa[:, row] = sc.T
    return dD, sa, dw
