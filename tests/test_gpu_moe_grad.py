"""GPU tests of the expert sort, its gradient, the gradient of the combine and
the masked dispatch, against the CPU oracle's layout and quantiser and plain
NumPy.  Positions, moved rows, codes, scales and products with one rounding
must match bit for bit; sums carry the bound of their order."""
import numpy as np
import pytest
import torch

import oracle
from fp8_block_scaled_x128_b200 import synth

from .parity_util import assert_close, bf16_to_f64
from .test_gpu_moe import routing, tokens

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from fp8_block_scaled_x128_b200 import gemm
    gemm.device_error(clear=True)
    return gemm


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def blocks_for(T, topk, G):
    return (T * topk + 127) // 128 + G


SHAPES = [  # T, topk, G, N, drop
    (1, 1, 1, 8, 0.0), (1, 8, 16, 7168, 0.0), (300, 2, 5, 384, 0.1), (129, 3, 7, 520, 0.2), (2500, 6, 256, 256, 0.0),
    (200, 12, 16, 128, 0.3), (40, 16, 200, 2112, 0.05), (9000, 4, 9, 64, 0.02), (33000, 1, 3, 8, 0.0),
    (1187, 16, 40, 128, 0.1), (2001, 8, 32, 640, 0.05), (1185, 2, 5, 384, 0.0), (4099, 3, 6, 1024, 0.0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,topk,G,N,drop", SHAPES)
def test_permute_and_its_gradient(g, T, topk, G, N, drop, dtype):
    e = routing(T + G, T, topk, G, drop) if topk <= G else routing(0, T, topk, G, drop, skew=0)
    x = tokens(T + N, T, N)
    nb = blocks_for(T, topk, G)
    used, cnt, off, pos, mi = oracle.moe_layout(e, G, nb)
    xs = torch.full((nb * 128, N), -5.0, dtype=dtype, device="cuda")
    out = (xs, torch.empty(T * topk, dtype=torch.int32, device="cuda"), torch.empty(nb, dtype=torch.int32, device="cuda"))
    xs, p, m = g.moe_permute(cuda(x, dtype), cuda(e), topk, G, out=out)
    assert np.array_equal(host(p), pos) and np.array_equal(host(m), mi)
    want = np.full((nb * 128, N), -5.0, np.float32)
    want[:used * 128] = 0
    live = pos >= 0
    want[pos[live]] = x[np.nonzero(live)[0] // topk]
    assert np.array_equal(host(xs), want)
    # the gradient: FP32 sum in slot order, one rounding
    d = synth.round_to_bf16(np.random.default_rng(T).standard_normal((nb * 128, N)).astype(np.float32))
    dx = g.moe_permute_backward(cuda(d, dtype), p, T, topk)
    acc = np.zeros((T, N), np.float32)
    for k in range(topk):
        q = pos.reshape(T, topk)[:, k]
        acc[q >= 0] += d[q[q >= 0]]
    assert np.array_equal(host(dx), synth.round_to_bf16(acc) if dtype == torch.bfloat16 else acc)
    # <permute(x), d> == <x, gradient(d)>: exact adjoint, in 64 bits, over the routed rows
    lhs = float((want[pos[live]].astype(np.float64) * d[pos[live]]).sum())
    rhs = float((x.astype(np.float64) * acc).sum())
    mags = float(np.abs(want[pos[live]].astype(np.float64) * d[pos[live]]).sum())
    assert abs(lhs - rhs) <= topk * U * mags + 1e-12 * mags
    assert g.device_error() == 0


def test_permute_of_no_tokens_and_of_dropped_ones(g):
    x = torch.zeros(0, 64, device="cuda")
    _, p, m = g.moe_permute(x, torch.zeros(0, dtype=torch.int32, device="cuda"), 4, 6)
    assert p.numel() == 0 and host(m).tolist() == [-1] * 6
    xs = torch.full((128 * 7, 64), 3.0, device="cuda")
    e = torch.full((10,), -1, dtype=torch.int32, device="cuda")
    xs, p, m = g.moe_permute(torch.ones(5, 64, device="cuda"), e, 2, 6,
                             out=(xs, torch.empty(10, dtype=torch.int32, device="cuda"),
                                  torch.empty(7, dtype=torch.int32, device="cuda")))
    assert bool((xs == 3).all()) and bool((p == -1).all()) and bool((m == -1).all())
    dx = g.moe_permute_backward(xs, p, 5, 2)
    assert bool((dx == 0).all())
    dD = torch.full((128 * 7, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((10,), 9.0, device="cuda")
    g.moe_combine_backward(torch.ones(5, 64, dtype=torch.bfloat16, device="cuda"), dD.clone(), p,
                           torch.ones(10, device="cuda"), 5, 2, out=(dD, dw))
    assert bool((dD == 3).all()) and bool((dw == 0).all())
    assert g.device_error() == 0


@pytest.mark.parametrize("T,topk,G,N,drop", [s for s in SHAPES if s[3] <= 2112 or s[0] == 1])
def test_combine_backward_rows_and_weights(g, T, topk, G, N, drop):
    rng = np.random.default_rng(T + N)
    e = routing(T + G, T, topk, G, drop) if topk <= G else routing(0, T, topk, G, drop, skew=0)
    nb = blocks_for(T, topk, G)
    used, cnt, off, pos, mi = oracle.moe_layout(e, G, nb)
    dout, D = tokens(1, T, N), tokens(2, nb * 128, N)
    w = rng.standard_normal(T * topk).astype(np.float32)
    w[::7] = 0
    live = pos >= 0
    tok = np.nonzero(live)[0] // topk
    prod = w[live, None] * dout[tok]                      # one FP32 product
    doutd, Dd, pd, wd = cuda(dout, torch.bfloat16), cuda(D, torch.bfloat16), cuda(pos), cuda(w)
    dD = torch.full((nb * 128, N), -5.0, dtype=torch.bfloat16, device="cuda")
    dD, dw = g.moe_combine_backward(doutd, Dd, pd, wd, T, topk, out=(dD, torch.empty(T * topk, device="cuda")))
    want = np.full((nb * 128, N), -5.0, np.float32)
    want[:used * 128] = 0
    want[pos[live]] = synth.round_to_bf16(prod)
    assert np.array_equal(host(dD), want)
    # a thread adds 8 products per 2048 columns, then two butterflies: at most
    # 8 ceil(N / 2048) + 20 roundings on a term
    terms = dout[tok].astype(np.float64) * D[pos[live]]
    ref = np.zeros(T * topk)
    ref[live] = terms.sum(1)
    lim = np.zeros(T * topk)
    lim[live] = (8 * -(-N // 2048) + 20) * U * np.abs(terms).sum(1)
    assert np.all(np.abs(host(dw) - ref) <= lim)
    # weights of one
    one, none = g.moe_combine_backward(doutd, Dd, pd, None, T, topk, out=(torch.zeros_like(dD), None))
    assert none is None and np.array_equal(host(one)[pos[live]], dout[tok])
    if N % 128 == 0:
        q = torch.full((nb * 128, N), 0x5A, dtype=torch.uint8, device="cuda")
        sa = torch.full((N // 128, nb * 128), -5.0, device="cuda")
        q, sa, dw2 = g.moe_combine_backward(doutd, Dd, pd, wd, T, topk, quantize=True,
                                            out=(q, sa, torch.empty_like(dw)))
        eq, esa = oracle.quantize_1x128(np.ascontiguousarray(prod)) if live.any() else (None, None)
        wq, ws = np.full((nb * 128, N), 0x5A, np.uint8), np.full((N // 128, nb * 128), -5.0, np.float32)
        wq[:used * 128], ws[:, :used * 128] = 0, 0
        if live.any():
            wq[pos[live]], ws[:, pos[live]] = eq, esa[:, :len(tok)]
        assert np.array_equal(host(sa), ws) and np.array_equal(host(q), wq)
        assert torch.equal(dw2, dw)
    assert g.device_error() == 0


def test_codes_of_tiny_and_huge_values(g):
    """Groups far below and above 1, subnormal products and scales, zeros of both
    signs: codes and scales of the definition, bit for bit."""
    T, topk, N = 24, 3, 384
    rng = np.random.default_rng(7)
    x = tokens(8, T, N)
    x[:, ::5] = 0
    x[:, 1::5] = -0.0
    x[3] = 0
    w = np.array([1, -1, 0, 1e-30, 1e-38, 1e-42, 1.4e-45, 1e30, 3e36, -2.5, 1e-25, 8e-25], np.float32)[
        rng.integers(0, 12, T * topk)]
    pos = rng.permutation(256)[:T * topk].astype(np.int32)
    prod = w[:, None] * synth.round_to_bf16(x)[np.arange(T * topk) // topk]
    assert np.isfinite(prod).all()
    eq, es = oracle.quantize_1x128(np.ascontiguousarray(prod))
    # w = 1.4e-45 (2^-149): |prod| <= 2^-146, and 2^-146 / 448 < 2^-150 rounds to a
    # scale of zero, where the definition divides by zero; such a group counts as
    # all-zero: scale 1, zero codes with the values' signs
    gone = es[:, :T * topk].T == 0
    assert gone.any() and np.abs(prod).reshape(T * topk, -1, 128).max(-1)[gone].max() <= 2.0 ** -146
    es[:, :T * topk][gone.T] = 1
    eq = np.where(np.repeat(gone, 128, 1), np.signbit(prod) * np.uint8(0x80), eq)
    D = torch.zeros(256, N, dtype=torch.bfloat16, device="cuda")
    q, sa, _ = g.moe_combine_backward(cuda(x, torch.bfloat16), D, cuda(pos), cuda(w), T, topk, quantize=True)
    assert np.array_equal(host(sa)[:, pos], es[:, :T * topk]) and np.array_equal(host(q)[pos], eq)
    for scale in (1e-38, 1e-30, 1e-20, 1.0, 1e30):
        xs = (x * np.float32(scale)).astype(np.float32)
        e = rng.integers(0, 4, T * topk).astype(np.int32)
        A, s, p, m = g.moe_dispatch_masked(cuda(xs), cuda(e), topk, 4, T * topk)
        wp, wm, wq, ws, _ = masked_reference(xs, e, topk, 4, T * topk)
        assert np.array_equal(host(p), wp)
        tok = np.arange(T * topk) // topk
        assert np.array_equal(host(A).reshape(-1, N)[wp], wq[tok])
        assert np.array_equal(host(s)[wp // (T * topk), :, wp % (T * topk)], ws[:, tok].T)
    assert g.device_error() == 0


def test_bad_positions_are_flagged_and_skipped(g):
    T, topk, N = 6, 2, 128
    pos = np.array([0, 1, 128, 3, -9, 4, 127, 5, 1 << 30, 6, -1, 7], np.int32)   # 128, -9 and 2^30 are no rows
    ok = np.where((pos >= 0) & (pos < 128), pos, -1)
    d = tokens(3, 128, N)
    g.device_error(clear=True)
    dx = g.moe_permute_backward(cuda(d), cuda(pos), T, topk)
    assert g.device_error() == g.DEVERR_BAD_POS
    want = np.zeros((T, N), np.float32)
    for r, p in enumerate(ok):
        if p >= 0:
            want[r // topk] += d[p]
    assert np.array_equal(host(dx), want)
    dout = cuda(tokens(4, T, N), torch.bfloat16)
    w = torch.ones(T * topk, device="cuda")
    dD, dw = g.moe_combine_backward(dout, cuda(d, torch.bfloat16), cuda(pos), w, T, topk)
    assert g.device_error() == g.DEVERR_BAD_POS
    assert np.array_equal(host(dD)[ok[ok >= 0]], host(dout)[np.nonzero(ok >= 0)[0] // topk])
    assert np.all(host(dw)[ok < 0] == 0)
    twice = np.where(np.arange(12) < 2, 5, -1).astype(np.int32)
    g.moe_combine_backward(dout, cuda(d, torch.bfloat16), cuda(twice), w, T, topk)
    assert g.device_error() == g.DEVERR_BAD_POS
    # bad experts: dropped and flagged, as in the quantised dispatch
    e = np.array([0, 3, -2, 1, 7, 2, 0, 0, 1, 1, 2, -1], np.int32)
    _, p, _ = g.moe_permute(cuda(tokens(5, T, N)), cuda(e), topk, 3)
    assert g.device_error() == g.DEVERR_BAD_EXPERT
    want = oracle.moe_layout(np.where((e < 0) | (e > 2), -1, e).astype(np.int32), 3, 4)[3]
    assert np.array_equal(host(p), want)


def masked_reference(x, e, topk, G, Mmax):
    pos = np.full(e.size, -1, np.int32)
    cnt = np.zeros(G, np.int64)
    for r, ex in enumerate(e):
        if 0 <= ex < G:
            if cnt[ex] < Mmax:
                pos[r] = ex * Mmax + cnt[ex]
            cnt[ex] += 1
    q, s = oracle.quantize_1x128(x)
    return pos, np.minimum(cnt, Mmax).astype(np.int32), q, s, bool((cnt > Mmax).any())


MASKED = [  # T, topk, G, K, Mmax, drop
    (1, 1, 1, 128, 4, 0.0), (1, 8, 16, 7168, 256, 0.0), (64, 8, 16, 384, 64, 0.1), (37, 3, 7, 2048, 40, 0.2),
    (200, 4, 8, 256, 20, 0.0), (256, 16, 256, 128, 256, 0.0), (700, 6, 33, 128, 700, 0.05), (1100, 4, 64, 640, 50, 0.0),
    (6000, 2, 3, 128, 6000, 0.01),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,topk,G,K,Mmax,drop", MASKED)
def test_dispatch_masked_matches_oracle(g, T, topk, G, K, Mmax, drop, dtype):
    x = tokens(T + K, T, K)
    e = routing(T + G, T, topk, G, drop)
    pos, mm, q, s, over = masked_reference(x, e, topk, G, Mmax)
    ld = (Mmax + 3) // 4 * 4 + 4
    out = (torch.full((G, Mmax, K), 0x5A, dtype=torch.uint8, device="cuda"),
           torch.full((G, K // 128, ld), -5.0, device="cuda"), torch.empty(T * topk, dtype=torch.int32, device="cuda"),
           torch.empty(G, dtype=torch.int32, device="cuda"))
    g.device_error(clear=True)
    A, sa, p, m = g.moe_dispatch_masked(cuda(x, dtype), cuda(e), topk, G, Mmax, out=out)
    assert np.array_equal(host(p), pos) and np.array_equal(host(m), mm)
    wA, ws = np.full((G * Mmax, K), 0x5A, np.uint8), np.full((G, K // 128, ld), -5.0, np.float32)
    live = pos >= 0
    tok = np.nonzero(live)[0] // topk
    wA[pos[live]] = q[tok]
    ws[pos[live] // Mmax, :, pos[live] % Mmax] = s[:, tok].T
    assert np.array_equal(host(A).reshape(G * Mmax, K), wA) and np.array_equal(host(sa), ws)
    assert g.device_error() == (g.DEVERR_MASKED_OVER if over else 0)


def test_dispatch_masked_of_repeated_bad_and_no_experts(g):
    x = tokens(1, 50, 128)
    e = np.full(50 * 4, 2, np.int32)                        # one expert four times in every token
    pos, mm, *_ = masked_reference(x, e, 4, 3, 300)
    _, _, p, m = g.moe_dispatch_masked(cuda(x), cuda(e), 4, 3, 300)
    assert np.array_equal(host(p), pos) and np.array_equal(host(m), mm) and g.device_error() == 0
    e[[0, 9]] = [3, -5]
    pos, mm, *_ = masked_reference(x, e, 4, 3, 300)
    _, _, p, m = g.moe_dispatch_masked(cuda(x), cuda(e), 4, 3, 300)
    assert np.array_equal(host(p), pos) and np.array_equal(host(m), mm)
    assert g.device_error() == g.DEVERR_BAD_EXPERT
    _, _, p, m = g.moe_dispatch_masked(torch.zeros(0, 128, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                                       4, 3, 300)
    assert p.numel() == 0 and host(m).tolist() == [0, 0, 0]


def test_long_batches_with_bad_experts(g):
    """More slots than a warp of the layout kernel keeps in registers, some experts
    out of range: positions and counts of the oracle, flagged."""
    T, topk, G = 24000, 4, 37
    e = routing(6, T, topk, G, 0.01)
    e[[5, 4000, T * topk - 1]] = [G, -3, 1 << 20]
    clean = np.where((e < 0) | (e >= G), -1, e).astype(np.int32)
    x = tokens(3, T, 128)
    xs, pos, mi = g.moe_permute(cuda(x), cuda(e), topk, G)
    assert g.device_error() == g.DEVERR_BAD_EXPERT
    used, cnt, off, wp, wm = oracle.moe_layout(clean, G, mi.numel())
    assert np.array_equal(host(pos), wp) and np.array_equal(host(mi), wm)
    live = wp >= 0
    assert np.array_equal(host(xs)[wp[live]], x[np.nonzero(live)[0] // topk])
    Mmax = int(np.bincount(clean[clean >= 0], minlength=G).max()) - 5          # some experts overflow
    A, sa, pos, mm = g.moe_dispatch_masked(cuda(x), cuda(e), topk, G, Mmax)
    assert g.device_error() == g.DEVERR_BAD_EXPERT | g.DEVERR_MASKED_OVER
    wp, wm, wq, _, over = masked_reference(x, clean, topk, G, Mmax)
    assert over and np.array_equal(host(pos), wp) and np.array_equal(host(mm), wm)
    live = wp >= 0
    assert np.array_equal(host(A).reshape(G * Mmax, 128)[wp[live]], wq[np.nonzero(live)[0] // topk])


def test_rows_past_32_bit_offsets(g):
    """Layouts of more than 2^32 bytes and 2^31 elements: the rows at their end."""
    T, topk, G, N = 34000, 8, 16, 8192
    e = cuda(routing(4, T, topk, G))
    x = torch.randn(T, N, device="cuda", dtype=torch.bfloat16)
    xs, pos, _ = g.moe_permute(x, e, topk, G)
    assert xs.numel() > 2 ** 31
    last = torch.arange(T * topk, device="cuda")[-4000:]
    assert int(pos.max()) * N > 2 ** 31
    high = torch.topk(pos, 4000).indices                  # the slots in the layout's last rows
    for sl in (last, high):
        assert torch.equal(xs[pos[sl].long()], x[sl // topk])
    w = torch.rand(T * topk, device="cuda")
    dx = g.moe_permute_backward(xs, pos, T, topk)
    assert torch.equal(dx[-500:], (x[-500:].float() * topk).to(torch.bfloat16))     # eight equal rows: exact
    dD, dw = g.moe_combine_backward(x, xs, pos, w, T, topk)
    assert torch.equal(dD[pos[high].long()], (w[high, None] * x[high // topk].float()).to(torch.bfloat16))
    want = (x[high // topk].double() ** 2).sum(1)
    assert bool(((dw[high].double() - want).abs() <= 60 * U * want).all())           # all terms positive
    del xs, dD, dx
    torch.cuda.empty_cache()
    G, Mmax, K = 256, 4200, 4096
    x = cuda(tokens(2, 9, K), torch.bfloat16)
    e = torch.tensor([255, 254, 0, 255, 3, 255, 255, 254, 1], dtype=torch.int32, device="cuda")
    A, sa, p, m = g.moe_dispatch_masked(x, e, 1, G, Mmax)
    assert A.numel() > 2 ** 32
    q, s = g.quantize_1x128(x)
    assert p.tolist() == [255 * Mmax, 254 * Mmax, 0, 255 * Mmax + 1, 3 * Mmax, 255 * Mmax + 2, 255 * Mmax + 3,
                          254 * Mmax + 1, Mmax]
    for t in range(9):
        grp, row = divmod(int(p[t]), Mmax)
        assert torch.equal(A[grp, row], q[t]) and torch.equal(sa[grp, :, row], s[:, t])
    assert g.device_error() == 0


def bf16_bits(t):
    torch.cuda.synchronize()
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("T", [1, 37])
def test_decode_block_in_a_graph(g, T):
    """norms -> masked dispatch -> masked GEMM -> combine -> norms of the next
    block, captured once and replayed on new tokens; every stage against the
    oracle or the 64-bit definition on what the stage before it gave."""
    from . import reference64 as ref
    from .test_gpu_norm import rounded, within
    H, topk, G, Mmax = 512, 2, 4, 64
    B, sb = synth.grouped_b(14, G, H, H)
    Bd, sbd = cuda(B), cuda(sb)
    y, h = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    e = torch.zeros(T * topk, dtype=torch.int32, device="cuda")
    w = torch.zeros(T * topk, device="cuda")
    gen = torch.Generator().manual_seed(T)
    post_w, pre_w = (1 + 0.2 * torch.randn(H, generator=gen) for _ in range(2))
    kw = dict(post_weight=post_w.cuda(), scale=0.5, pre_weight=pre_w.cuda(), eps=1e-6)
    A = torch.zeros(G, Mmax, H, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(G, H // 128, Mmax, device="cuda")
    pos = torch.empty(T * topk, dtype=torch.int32, device="cuda")
    mm = torch.empty(G, dtype=torch.int32, device="cuda")
    D = torch.zeros(G, Mmax, H, dtype=torch.bfloat16, device="cuda")

    def step():
        h1, z = g.norm_residual(y, h, **kw)
        g.moe_dispatch_masked(z, e, topk, G, Mmax, out=(A, sa, pos, mm))
        g.m_grouped_fp8_gemm_nt_masked(A, sa, Bd, sbd, mm, 16, D=D)
        out = g.moe_combine(D, pos, w, T, topk)
        return (h1, z, out, *g.norm_residual(out, h1, quantize=True, **kw))

    step()
    # that step sent every slot to expert 0: more than its Mmax rows for T = 37
    assert g.device_error() == (g.DEVERR_MASKED_OVER if T * topk > Mmax else 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h1, z, out, h2, q2, s2 = step()
    for turn in range(2):
        y.copy_(torch.randn(T, H, generator=gen))
        h.copy_(torch.randn(T, H, generator=gen))
        er = routing(turn, T, topk, G, 0.1 if T > 1 else 0.0)
        e.copy_(torch.from_numpy(er))
        w.copy_(torch.rand(T * topk, generator=gen))
        graph.replay()
        args = (y.cpu().double(), h.cpu().double(), post_w.double(), None, 0.5, pre_w.double(), float(np.float32(1e-6)))
        hp, zz, _ = ref.forward(*args)
        eh, ez = ref.forward_bounds(*args)
        within(h1, hp, rounded(hp, eh, torch.bfloat16), "h1")
        within(z, zz, rounded(zz, ez, torch.bfloat16), "z")
        wp, wm, wq, ws, _ = masked_reference(host(z), er, topk, G, Mmax)
        assert np.array_equal(host(pos), wp) and np.array_equal(host(mm), wm)
        for k, p in enumerate(wp):
            if p >= 0:
                assert np.array_equal(host(A).reshape(G * Mmax, H)[p], wq[k // topk])
        exact, _ = oracle.m_grouped_masked(host(A), host(sa), Mmax, B, sb, wm, G, Mmax, H, H)
        rows = wp[wp >= 0]
        assert_close(bf16_bits(D).reshape(G * Mmax, H)[rows], np.asarray(exact).reshape(G * Mmax, H)[rows], "D")
        want = oracle.moe_combine(bf16_bits(D).reshape(G * Mmax, H), wp, host(w), T, topk)
        assert np.array_equal(bf16_bits(out), want)
        args = (out.cpu().double(), h1.cpu().double(), *args[2:])
        hp, zz, _ = ref.forward(*args)
        eh, ez = ref.forward_bounds(*args)
        within(h2, hp, rounded(hp, eh, torch.bfloat16), "h2")
        # codes: half an e4m3 step of the quotient (2^-4, or 2^-10 below its normal range), the
        # error of z over the scale and that of the scale
        sc = s2.cpu().double().T[:T].repeat_interleave(128, 1)
        val = q2.view(torch.float8_e4m3fn).float().cpu().double() * sc
        within(val, zz, 2.0 ** -4 * zz.abs() * (1 + 1e-3) + sc * 2.0 ** -10 + 2 * ez, "codes")
    assert g.device_error() == 0


def test_training_block_forward_and_backward(g):
    """norms -> quantised dispatch -> grouped GEMM -> combine, and back: combine
    gradient (quantised) -> grouped GEMM with the transposed weights -> sort
    gradient -> norm gradient.  Each stage against the oracle or 64 bits on what
    the stage before it gave."""
    from . import reference64 as ref
    from .test_gpu_norm import rounded, within
    T, topk, G, H, N = 300, 2, 4, 512, 384
    gen = torch.Generator().manual_seed(21)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    y, h = rnd(T, H).to(torch.bfloat16).cuda(), rnd(T, H).to(torch.bfloat16).cuda()
    post_w, pre_w, gate = 1 + 0.2 * rnd(H), 1 + 0.2 * rnd(H), rnd(H)
    W = (rnd(G, N, H) * 0.05).to(torch.bfloat16).cuda()
    fwd = [g.quantize_128x128(W[i].contiguous()) for i in range(G)]
    bwd = [g.quantize_128x128(W[i].T.contiguous()) for i in range(G)]
    B, sb = torch.stack([a for a, _ in fwd]), torch.stack([b for _, b in fwd])
    Bt, sbt = torch.stack([a for a, _ in bwd]), torch.stack([b for _, b in bwd])
    er = routing(5, T, topk, G, 0.05)
    e, w = cuda(er), torch.rand(T * topk, generator=gen).cuda()
    kw = dict(post_weight=post_w.cuda(), gate=gate.cuda(), scale=0.5, pre_weight=pre_w.cuda(), eps=1e-6)
    h1, z = g.norm_residual(y, h, **kw)
    A, sa, pos, mi = g.moe_dispatch(z, e, topk, G)
    D = g.m_grouped_fp8_gemm_nt_contiguous(A, sa, B, sb, mi)
    out = g.moe_combine(D, pos, w, T, topk)
    dout = rnd(T, N).to(torch.bfloat16).cuda()
    q, qs, dw = g.moe_combine_backward(dout, D, pos, w, T, topk, quantize=True)
    dA = g.m_grouped_fp8_gemm_nt_contiguous(q, qs, Bt, sbt, mi)
    dz = g.moe_permute_backward(dA, pos, T, topk)
    dh_out = rnd(T, H).to(torch.bfloat16).cuda()
    dh, dy, dpre, dpost, dgate = g.norm_residual_backward(dz, dh_out, h1, y, **kw)
    # forward
    used, eA, esa, epos, emi = oracle.moe_dispatch(host(z), er, topk, G, mi.numel())
    assert np.array_equal(host(pos), epos) and np.array_equal(host(mi), emi)
    M, rows = mi.numel() * 128, used * 128
    ex, _ = oracle.m_grouped_contiguous(eA, esa, esa.shape[1], host(B), host(sb), emi, M, N, H, G)
    assert_close(bf16_bits(D)[:rows], ex[:rows], "D")
    assert np.array_equal(bf16_bits(out), oracle.moe_combine(bf16_bits(D), epos, host(w), T, topk))
    # backward
    live = epos >= 0
    prod = host(w)[live, None] * host(dout)[np.nonzero(live)[0] // topk]
    eq, es = oracle.quantize_1x128(np.ascontiguousarray(prod))
    assert np.array_equal(host(q)[epos[live]], eq) and np.array_equal(host(qs)[:, epos[live]], es[:, :int(live.sum())])
    ref_dw = np.zeros(T * topk)
    terms = host(dout)[np.nonzero(live)[0] // topk].astype(np.float64) * bf16_to_f64(bf16_bits(D))[epos[live]]
    ref_dw[live] = terms.sum(1)
    lim = np.zeros(T * topk)
    lim[live] = 28 * U * np.abs(terms).sum(1)
    assert np.all(np.abs(host(dw) - ref_dw) <= lim)
    qz, sz = np.zeros((M, N), np.uint8), np.zeros((N // 128, M), np.float32)
    qz[epos[live]], sz[:, epos[live]] = eq, es[:, :int(live.sum())]
    ex, _ = oracle.m_grouped_contiguous(qz, sz, M, host(Bt), host(sbt), emi, M, H, N, G)
    assert_close(bf16_bits(dA)[:rows], ex[:rows], "dA")
    acc = np.zeros((T, H), np.float32)
    for k in range(topk):
        p = epos.reshape(T, topk)[:, k]
        acc[p >= 0] += host(dA)[p[p >= 0]]
    assert np.array_equal(host(dz), synth.round_to_bf16(acc))
    r = ref.backward(dz.cpu().double(), dh_out.cpu().double(), h1.cpu().double(), y.cpu().double(), post_w.double(),
                     gate.double(), 0.5, pre_w.double(), float(np.float32(1e-6)))
    for t, name, dt in ((dh, "dh", torch.bfloat16), (dy, "dy", torch.bfloat16), (dpre, "dpre", torch.float32),
                        (dpost, "dpost", torch.float32), (dgate, "dgate", torch.float32)):
        within(t, r[name], rounded(r[name], r["e_" + name], dt), name)
    assert g.device_error() == 0


def test_calls_on_other_streams_and_in_graphs(g):
    """The same operands on two streams at once, and captured calls replayed on
    new routings, give what plain calls give."""
    T, topk, G, N = 500, 4, 12, 1024
    x = cuda(tokens(1, T, N), torch.bfloat16)
    experts = [cuda(routing(i, T, topk, G, 0.1)) for i in range(3)]
    w = torch.rand(T * topk, device="cuda")
    nb = blocks_for(T, topk, G)

    def chain(e, stream=None):
        xs, pos, mi = g.moe_permute(x, e, topk, G, stream=stream)
        dD, dw = g.moe_combine_backward(x, xs, pos, w, T, topk, stream=stream)
        return pos, mi, dw, g.moe_permute_backward(dD, pos, T, topk, stream=stream)

    want = [chain(e) for e in experts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [chain(e, s) for e, s in zip(experts, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for r, q in zip(want, got) for a, b in zip(r, q))
    e = experts[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(e)
    for i in (1, 2, 0):
        e.copy_(experts[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[i], got))
    assert nb * 128 >= T * topk and g.device_error() == 0


def test_slots_in_the_shape_of_the_router(g):
    """Experts and positions as [T, topk] tensors give what flat ones give."""
    T, topk, G, N = 70, 3, 5, 256
    x, e = cuda(tokens(6, T, N), torch.bfloat16), cuda(routing(7, T, topk, G, 0.1))
    xs, pos, mi = g.moe_permute(x, e, topk, G)
    xs2, pos2, mi2 = g.moe_permute(x, e.view(T, topk), topk, G)
    used = int((mi >= 0).sum()) * 128
    assert torch.equal(xs[:used], xs2[:used]) and torch.equal(pos, pos2) and torch.equal(mi, mi2)
    assert torch.equal(g.moe_permute_backward(xs, pos, T, topk), g.moe_permute_backward(xs, pos.view(T, topk), T, topk))
    w = torch.rand(T * topk, device="cuda")
    for a, b in zip(g.moe_combine_backward(x, xs, pos, w, T, topk), g.moe_combine_backward(x, xs, pos.view(T, topk), w, T, topk)):
        assert torch.equal(a[:used], b[:used])
    a, b = (g.moe_dispatch_masked(x, s, topk, G, 128) for s in (e, e.view(T, topk)))
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
    A, B = a[0].view(-1, N), b[0].view(-1, N)
    live = a[2][a[2] >= 0].long()
    assert torch.equal(A[live], B[live]) and g.device_error() == 0
