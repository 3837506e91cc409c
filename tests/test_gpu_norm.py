"""GPU tests of fp8g_norm_residual and fp8g_norm_residual_backward against the
64-bit definitions (tests/reference64.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

import oracle

from . import reference64 as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from fp8_block_scaled_x128_b200 import gemm
    gemm.device_error(clear=True)
    return gemm


def inputs(seed, rows, H, dtype, post, gate, res, pre):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    x = dict(y=(rnd(rows, H) * 0.7).to(dtype), h=rnd(rows, H).to(dtype) if res else None,
             post_w=1 + 0.3 * rnd(H) if post else None, pre_w=1 + 0.3 * rnd(H) if pre else None,
             gate={"none": None, "channel": rnd(H), "token": rnd(rows, 1)}[gate], scale=0.37)
    return x, gen


def dev(t):
    return None if t is None else t.cuda()


def dbl(t):
    return None if t is None else t.cpu().double()


def call(g, x, **kw):
    return g.norm_residual(dev(x["y"]), dev(x["h"]), post_weight=dev(x["post_w"]), gate=dev(x["gate"]),
                           scale=x["scale"], pre_weight=dev(x["pre_w"]), eps=EPS, **kw)


def args64(x):
    # the scale reaches the kernel as FP32
    return (dbl(x["y"]), dbl(x["h"]), dbl(x["post_w"]), dbl(x["gate"]), float(np.float32(x["scale"])), dbl(x["pre_w"]),
            float(np.float32(EPS)))


def within(got, want, bound, what):
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst by {float((err - bound).max()):.3g}"


def rounded(want, bound, dtype):
    """The bound after the final rounding to dtype."""
    return bound + ref.ROUND[dtype] * (want.abs() + bound) + 1e-38


CASES = [  # rows, H, post, gate, residual, pre-weight
    (1, 7168, True, "none", True, True), (1, 8, True, "channel", True, True), (5, 8, False, "none", False, False),
    (3, 256, False, "channel", True, True), (64, 512, True, "token", True, True), (37, 2112, True, "channel", False, True),
    (130, 1000, True, "token", True, False), (300, 4096, True, "channel", True, True), (7, 8192, True, "channel", True, True),
    (5, 8200, True, "channel", True, True), (3, 16384, True, "token", True, True), (700, 136, True, "channel", True, True),
    (5000, 64, True, "none", True, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,H,post,gate,res,pre", CASES)
def test_forward_matches_the_definition(g, rows, H, post, gate, res, pre, dtype):
    x, _ = inputs(rows + H, rows, H, dtype, post, gate, res, pre)
    h_out, z = call(g, x)
    hp, zz, _ = ref.forward(*args64(x))
    eh, ez = ref.forward_bounds(*args64(x))
    within(h_out, hp, rounded(hp, eh, dtype), "h_out")
    within(z, zz, rounded(zz, ez, dtype), "z")
    assert g.device_error() == 0


@pytest.mark.parametrize("rows,H,post,gate", [(1, 7168, True, "none"), (5, 128, True, "channel"), (33, 1152, False, "none"),
                                              (9, 8192, True, "token"), (3, 16384, True, "channel"), (2, 8320, True, "none"),
                                              (400, 640, True, "channel")])
def test_quantised_output_is_the_quantiser_of_z(g, rows, H, post, gate):
    """FP32 rows: z is stored unrounded, so the fused codes and scales must be
    bit for bit what the quantiser's definition makes of it; bf16 rows: the same
    through a call on the widened inputs."""
    x, _ = inputs(rows + H + 1, rows, H, torch.float32, post, gate, True, True)
    x["y"][:, 128 * (H // 256):128 * (H // 256) + 128] = 0     # h alone in one group
    x["h"][0, :128] = 0
    x["y"][0, :128] = 0                                        # an all-zero group
    for dtype in (torch.float32, torch.bfloat16):
        xs = dict(x, y=x["y"].to(dtype), h=x["h"].to(dtype))
        wide = dict(x, y=xs["y"].float(), h=xs["h"].float())
        _, z = call(g, wide)
        h_out, q, sa = call(g, xs, quantize=True)
        eq, esa = oracle.quantize_1x128(z.cpu().numpy(), ld_sa=sa.shape[1])
        assert np.array_equal(sa.cpu().numpy()[:, :rows], esa[:, :rows])
        assert np.array_equal(q.cpu().numpy(), eq)
        assert torch.equal(h_out, call(g, xs)[0])


@pytest.mark.parametrize("size", [1e-36, 1e-24, 1e-10, 1e12])
def test_quantised_tiny_and_huge_rows(g, size):
    """Pre-weights that bring z near either end of FP32: the fused codes are
    still the quantiser's of the FP32 z."""
    x, _ = inputs(17, 9, 640, torch.float32, True, "channel", True, True)
    x["pre_w"] *= size
    x["pre_w"][::7] = -0.0
    _, z = call(g, x)
    _, q, sa = call(g, x, quantize=True)
    eq, esa = oracle.quantize_1x128(z.cpu().numpy(), ld_sa=sa.shape[1])
    assert np.array_equal(sa.cpu().numpy()[:, :9], esa[:, :9]) and np.array_equal(q.cpu().numpy(), eq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,H,post,gate,res,pre", CASES)
def test_backward_matches_the_formulas(g, rows, H, post, gate, res, pre, dtype):
    x, gen = inputs(rows + 3 * H, rows, H, dtype, post, gate, True, pre)
    dz, dho = (torch.randn(rows, H, generator=gen).to(dtype) for _ in range(2))
    for dz_, dho_ in ((dz, dho), (dz, None), (None, dho)) if H <= 1000 else ((dz, dho),):
        got = g.norm_residual_backward(dev(dz_), dev(dho_), dev(x["h"]), dev(x["y"]), post_weight=dev(x["post_w"]),
                                       gate=dev(x["gate"]), scale=x["scale"], pre_weight=dev(x["pre_w"]), eps=EPS)
        y, hp, post_w, gt, s, pre_w, eps = args64(x)
        r = ref.backward(dbl(dz_), dbl(dho_), hp, y, post_w, gt, s, pre_w, eps)
        within(got[0], r["dh"], rounded(r["dh"], r["e_dh"], dtype), "dh")
        within(got[1], r["dy"], rounded(r["dy"], r["e_dy"], dtype), "dy")
        for t, name in zip(got[2:], ("dpre", "dpost", "dgate")):
            assert (t is None) == (r[name] is None), name
            if t is not None:
                assert t.shape == r[name].shape
                within(t, r[name], rounded(r[name], r["e_" + name], torch.float32), name)


def test_backward_agrees_with_differences_of_the_forward(g):
    """Central differences of <z, a> + <h', b> along a random direction of all
    inputs, FP32 on the GPU.  The bound: the forward's own error (at most 40 U
    of every term, twice, over the step), the gradients' own, and the
    truncation, which the same difference in 64 bits gives exactly."""
    rows, H = 23, 520
    x, gen = inputs(5, rows, H, torch.float32, True, "channel", True, True)
    rnd = lambda t: torch.randn(t.shape, generator=gen)
    a, b = rnd(x["y"]), rnd(x["y"])
    names = ("y", "h", "post_w", "gate", "pre_w")
    d = {n: rnd(x[n]) for n in names}
    step = 2.0 ** -7

    def moved(s):
        return dict(x, **{n: x[n] + s * d[n] for n in names})   # the FP32 values that both sides get

    def loss(hp, z):
        return float((z.cpu().double() * a.double()).sum() + (hp.cpu().double() * b.double()).sum())

    plus, minus = moved(step), moved(-step)
    fd = (loss(*call(g, plus)) - loss(*call(g, minus))) / (2 * step)
    fd64 = (loss(*ref.forward(*args64(plus))[:2]) - loss(*ref.forward(*args64(minus))[:2])) / (2 * step)
    h_out, _ = call(g, x)
    grads = g.norm_residual_backward(a.cuda(), b.cuda(), h_out, dev(x["y"]), post_weight=dev(x["post_w"]),
                                     gate=dev(x["gate"]), scale=x["scale"], pre_weight=dev(x["pre_w"]), eps=EPS)
    dh, dy, dpre, dpost, dgate = (t.cpu().double() for t in grads)
    dot = sum(float((t * d[n].double()).sum()) for t, n in ((dy, "y"), (dh, "h"), (dpost, "post_w"), (dgate, "gate"), (dpre, "pre_w")))
    hp, z, _ = ref.forward(*args64(x))
    rounding = 40 * ref.U * float((z * a.double()).abs().sum() + (hp * b.double()).abs().sum()) / step
    y64, _, post_w, gate, s, pre_w, eps = args64(x)
    r = ref.backward(a.double(), b.double(), dbl(h_out), y64, post_w, gate, s, pre_w, eps)
    pairs = (("dy", "y"), ("dh", "h"), ("dpost", "post_w"), ("dgate", "gate"), ("dpre", "pre_w"))
    terms = torch.cat([(r[k] * d[n].double()).flatten() for k, n in pairs])
    slack = sum(float((rounded(r[k], r["e_" + k], torch.float32) * d[n].double().abs()).sum()) for k, n in pairs)
    truncation = abs(fd64 - float(terms.sum()))     # both sides in 64 bits
    assert truncation <= 0.02 * float(terms.norm())
    assert abs(fd - dot) <= 2 * rounding + truncation + slack, (fd, dot, rounding, truncation, slack)


def test_zero_rows_and_zero_values(g):
    e = torch.empty(0, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    h_out, z = g.norm_residual(e, e, post_weight=w, pre_weight=w)
    assert h_out.shape == z.shape == (0, 256)
    dh, dy, dpre, dpost, dgate = g.norm_residual_backward(e, e, e, e, post_weight=w, pre_weight=w, gate=w)
    assert dh.shape == (0, 256) and float(dpre.abs().max()) == float(dpost.abs().max()) == float(dgate.abs().max()) == 0
    z0 = torch.zeros(4, 256, device="cuda")
    h_out, z = g.norm_residual(z0, z0, post_weight=w, pre_weight=w)
    assert float(h_out.abs().max()) == 0 and float(z.abs().max()) == 0
    got = g.norm_residual_backward(z0, z0 + 1, z0, z0, post_weight=w, pre_weight=w)
    assert all(bool(torch.isfinite(t).all()) for t in got if t is not None)
    # a closed gate per token: dy is 0, its gate's gradient is not
    x, gen = inputs(8, 6, 256, torch.float32, True, "token", True, True)
    x["gate"][2] = 0
    r = g.norm_residual_backward(torch.randn(6, 256, generator=gen).cuda(), None, dev(x["h"]), dev(x["y"]),
                                 post_weight=dev(x["post_w"]), gate=dev(x["gate"]), scale=1.0, pre_weight=dev(x["pre_w"]))
    assert float(r[1][2].abs().max()) == 0 and float(r[4][2]) != 0


def test_not_a_number_stays_in_its_row(g):
    x, _ = inputs(9, 5, 512, torch.bfloat16, True, "channel", True, True)
    x["y"][1, 7], x["h"][3, 500] = float("nan"), float("inf")
    h_out, z = call(g, x)
    clean = [0, 2, 4]
    assert bool(torch.isfinite(h_out[clean].float()).all()) and bool(torch.isfinite(z[clean].float()).all())
    assert bool(torch.isnan(z[1].float()).all()) and bool(torch.isnan(z[3, 500].float()))


def test_in_place_streams_and_graphs(g):
    """h_out may be h and z may be y; a call on another stream; the backward pass
    captured once and replayed on new inputs gives what a plain call gives."""
    x, gen = inputs(11, 300, 2112, torch.bfloat16, True, "channel", True, True)
    want = call(g, x)
    y, h = dev(x["y"]), dev(x["h"])
    kw = dict(post_weight=dev(x["post_w"]), gate=dev(x["gate"]), scale=x["scale"], pre_weight=dev(x["pre_w"]), eps=EPS)
    g.norm_residual(y, h, out=(h, y), **kw)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    side = torch.cuda.Stream()
    yy, hh = dev(x["y"]), dev(x["h"])
    torch.cuda.synchronize()
    got = g.norm_residual(yy, hh, stream=side, **kw)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dz, dho = (torch.randn(300, 2112, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    first = g.norm_residual_backward(dz, dho, want[0], yy, **kw)
    out = tuple(torch.empty_like(t) for t in first)
    ws = torch.empty(g.lib.fp8g_norm_residual_backward_workspace_bytes(300, 2112) // 4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.norm_residual_backward(dz, dho, want[0], yy, out=out, workspace=ws, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    dz.copy_(torch.randn(300, 2112, generator=gen))
    second = g.norm_residual_backward(dz, dho, want[0], yy, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(second, out))
    # dh over dh_out
    over = dho.clone()
    g.norm_residual_backward(dz, over, want[0], yy, out=(over, *out[1:]), **kw)
    assert torch.equal(over, second[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [128, 1152, 2112, 6152, 8192, 8320, 12416, 16384])
@pytest.mark.parametrize("post,gate", [(True, "token"), (False, "token"), (True, "channel"), (False, "none")])
def test_a_row_comes_out_alike_wherever_it_stands(g, H, post, gate, dtype):
    """Many rows a CTA or cluster, one after the other, give what each row gives
    in a call of few rows (a row each): every row's sums run in one order.  The
    first row of a CTA, its last ones and rows behind an infinite one included."""
    rows, part = 2 * 148 * 4 + 5 if H < 4096 else 601, 60
    x, gen = inputs(H, rows, H, dtype, post, gate, True, True)
    dz, dho = (torch.randn(rows, H, generator=gen).to(dtype).cuda() for _ in range(2))
    y, h, gt, w, pw = (dev(x[n]) for n in ("y", "h", "gate", "post_w", "pre_w"))
    y[11, 3] = float("inf")

    def run(at):
        kw = dict(post_weight=w, scale=x["scale"], pre_weight=pw, eps=EPS, gate=gt[at].contiguous() if gate == "token" else gt)
        h_out, z = g.norm_residual(y[at], h[at], **kw)
        dh, dy, _, _, dg = g.norm_residual_backward(dz[at], dho[at], h[at], y[at], **kw)
        out = [h_out, z, dh, dy] + ([dg] if gate == "token" else [])
        if H % 128 == 0:
            _, q, sa = g.norm_residual(y[at], h[at], quantize=True, **kw)
            out += [q, sa[:, :q.shape[0]].t()]
        return out

    bits = lambda t: t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])
    whole, clean = run(slice(None)), torch.arange(rows) != 11
    for r in (0, 300, rows - part):
        few = run(slice(r, r + part))
        for i, (a, b) in enumerate(zip(whole, few)):
            assert torch.equal(bits(a[r:r + part])[clean[r:r + part]], bits(b)[clean[r:r + part]]), (r, i)
    assert g.device_error() == 0


@pytest.mark.parametrize("H", [256, 7168, 12000])
def test_calls_at_once_on_two_streams_and_in_two_graphs(g, H):
    """Two backward passes under way together, each with the workspace it makes
    itself, and two captured ones replayed together, give what each gives alone."""
    rows = 700
    sides = []
    for seed in (1, 2):
        x, gen = inputs(seed, rows, H, torch.bfloat16, True, "channel", True, True)
        dz, dho = (torch.randn(rows, H, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
        y, h = dev(x["y"]), dev(x["h"])
        kw = dict(post_weight=dev(x["post_w"]), gate=dev(x["gate"]), scale=0.5, pre_weight=dev(x["pre_w"]), eps=EPS)
        sides.append((dz, dho, y, h, kw))

    def both(side, stream=None):
        dz, dho, y, h, kw = side
        h_out, z = g.norm_residual(y, h, stream=stream, **kw)
        return (h_out, z, *g.norm_residual_backward(dz, dho, h_out, y, stream=stream, **kw))

    want = [both(s) for s in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    for _ in range(5):
        got = [both(s, st) for s, st in zip(sides, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, q in zip(want, got) for a, b in zip(w, q))
    graphs, outs = [], []
    for s in sides:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(s))
        graphs.append(graph)
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, q in zip(want, outs) for a, b in zip(w, q))
    assert g.device_error() == 0


@pytest.mark.parametrize("H", [8192, 12288])
def test_rows_past_32_bit_offsets(g, H):
    """More than 2^31 elements: the rows behind that offset come out as in a call
    of their own, forward and backward."""
    rows = 2 ** 31 // H + 300
    gen = torch.Generator(device="cuda").manual_seed(3)
    y, h, dz = (torch.empty(rows, H, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    tail = slice(rows - 400, rows)
    for t in (y, h, dz):
        t[:400].normal_(generator=gen), t[400:-400].fill_(0.5), t[tail].normal_(generator=gen)
    w = 1 + 0.2 * torch.randn(H, device="cuda", generator=gen)
    kw = dict(post_weight=w, scale=0.5, pre_weight=w, eps=EPS)
    want = g.norm_residual(y[tail].contiguous(), h[tail].contiguous(), **kw)
    wq = g.norm_residual(y[tail].contiguous(), h[tail].contiguous(), quantize=True, **kw)
    wb = g.norm_residual_backward(dz[tail].contiguous(), None, h[tail].contiguous(), y[tail].contiguous(), **kw)
    got = g.norm_residual(y, h, **kw)
    assert torch.equal(got[0][tail], want[0]) and torch.equal(got[1][tail], want[1])
    del got
    _, q, sa = g.norm_residual(y, h, quantize=True, **kw)
    assert torch.equal(q[tail], wq[1]) and torch.equal(sa[:, tail], wq[2][:, :400])
    del q, sa
    dh, dy, _, _, _ = g.norm_residual_backward(dz, None, h, y, **kw)
    assert torch.equal(dh[tail], wb[0]) and torch.equal(dy[tail], wb[1])
    del dh, dy, y, h, dz
    torch.cuda.empty_cache()


def test_in_place_wide_rows(g):
    """h_out over h and z over y where a row takes a cluster of CTAs."""
    x, gen = inputs(19, 200, 12000, torch.float32, True, "token", True, True)
    want = call(g, x)
    y, h = dev(x["y"]), dev(x["h"])
    kw = dict(post_weight=dev(x["post_w"]), gate=dev(x["gate"]), scale=x["scale"], pre_weight=dev(x["pre_w"]), eps=EPS)
    g.norm_residual(y, h, out=(h, y), **kw)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    dz, dho = (torch.randn(200, 12000, generator=gen).cuda() for _ in range(2))
    first = g.norm_residual_backward(dz, dho, want[0], dev(x["y"]), **kw)
    over = dho.clone()
    g.norm_residual_backward(dz, over, want[0], dev(x["y"]), out=(over, *(torch.empty_like(t) for t in first[1:])), **kw)
    assert torch.equal(over, first[0])


def test_the_same_call_gives_the_same_bits(g):
    x, gen = inputs(12, 1500, 1024, torch.bfloat16, True, "channel", True, True)
    dz = torch.randn(1500, 1024, generator=gen).to(torch.bfloat16).cuda()
    kw = dict(post_weight=dev(x["post_w"]), gate=dev(x["gate"]), scale=1.0, pre_weight=dev(x["pre_w"]))
    h, y = dev(x["h"]), dev(x["y"])
    a = g.norm_residual_backward(dz, None, h, y, **kw)
    for _ in range(3):
        b = g.norm_residual_backward(dz, None, h, y, **kw)
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_parameters_beside_other_rows_stay_untouched(g):
    """Outputs are views between canaries: nothing is written beside them, and
    the scales' entries past the last row stay."""
    rows, H = 5, 384
    x, _ = inputs(13, rows, H, torch.bfloat16, True, "none", True, True)
    big = torch.full((rows + 2, H), -7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((rows + 2, H), 0x5A, dtype=torch.uint8, device="cuda")
    sa = torch.full((H // 128, 16), -3.0, device="cuda")
    call(g, x, quantize=True, out=(big[1:-1], q[1:-1], sa))
    assert bool((big[0] == -7).all()) and bool((big[-1] == -7).all())
    assert bool((q[0] == 0x5A).all()) and bool((q[-1] == 0x5A).all()) and bool((sa[:, rows:] == -3).all())
    assert bool((sa[:, :rows] > 0).all())


@pytest.mark.parametrize("H,most", [(1024, 8192), (4096, 1000), (12416, 700)])
def test_one_workspace_for_the_largest_batch(g, H, most):
    """The workspace of the largest batch serves smaller ones, whatever was left
    in it, and nothing is written behind it."""
    need = g.lib.fp8g_norm_residual_backward_workspace_bytes(most, H) // 4
    kept = torch.full((need + 64,), float("nan"), device="cuda")
    x, gen = inputs(most, most, H, torch.bfloat16, True, "channel", True, True)
    dz = torch.randn(most, H, generator=gen).to(torch.bfloat16).cuda()
    y, h = dev(x["y"]), dev(x["h"])
    kw = dict(post_weight=dev(x["post_w"]), gate=dev(x["gate"]), scale=0.5, pre_weight=dev(x["pre_w"]), eps=EPS)
    for rows in (most, most // 2 + 1, 592, 148, 1):
        if rows <= most:
            want = g.norm_residual_backward(dz[:rows], None, h[:rows], y[:rows], **kw)
            got = g.norm_residual_backward(dz[:rows], None, h[:rows], y[:rows], workspace=kept[:need], **kw)
            assert all(torch.equal(a, b) for a, b in zip(want, got)), rows
    assert bool(torch.isnan(kept[need:]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,H,post,gate", [(3001, 520, True, "channel"), (5003, 72, True, "channel"),
                                              (5003, 72, False, "channel"), (2777, 200, True, "token")])
def test_parameter_sums_of_many_rows(g, rows, H, post, gate, dtype):
    """More than 256 partial rows, added in two launches, with a last group of
    columns that is not full.  The bound counts the additions on one term's way: at
    most rows / 257 + 1 in its cluster, 4 in a warp and 32 over the warps in the first
    launch, 1 and 32 in the second, and 30 U for the term itself.  A row left out
    or taken twice would show: most of its terms are above the bound."""
    assert g.lib.fp8g_norm_residual_backward_workspace_bytes(rows, H) > 2 * 257 * H * 4
    x, gen = inputs(rows * H, rows, H, dtype, post, gate, True, True)
    dz, dho = (torch.randn(rows, H, generator=gen).to(dtype) for _ in range(2))
    got = g.norm_residual_backward(dev(dz), dev(dho), dev(x["h"]), dev(x["y"]), post_weight=dev(x["post_w"]),
                                   gate=dev(x["gate"]), scale=x["scale"], pre_weight=dev(x["pre_w"]), eps=EPS)
    y, hp, post_w, gt, s, pre_w, eps = args64(x)
    r = ref.backward(dbl(dz), dbl(dho), hp, y, post_w, gt, s, pre_w, eps)
    u = y * ref.rms_factor(y, eps) if post else y
    terms = {"dpre": (dbl(dz) * hp * ref.rms_factor(hp, eps), 0.0)}
    if post:
        terms["dpost"] = (s * gt * r["dh"] * u, (s * gt * u).abs() * r["e_dh"])
    if gate == "channel":
        w2 = post_w if post else torch.ones(1, dtype=torch.float64)
        terms["dgate"] = (s * w2 * r["dh"] * u, (s * w2 * u).abs() * r["e_dh"])
    for t, name in zip(got[2:], ("dpre", "dpost", "dgate")):
        if name not in terms:
            continue
        each, err = terms[name]
        bound = (rows // 257 + 70 + 30) * ref.U * each.abs().sum(0) + (err.sum(0) if torch.is_tensor(err) else err)
        shown = (each.abs() > 2 * bound).double().mean(1) > 0.5
        assert bool(shown.all()) if gate == "channel" else float(shown.double().mean()) > 0.9   # a token's gate may be near 0
        within(t, each.sum(0), rounded(each.sum(0), bound, torch.float32), name)
    assert g.device_error() == 0


@pytest.mark.parametrize("exchange", [0, 1])
@pytest.mark.parametrize("H,dtype", [(8200, torch.bfloat16), (12416, torch.bfloat16), (16384, torch.float32)],
                         ids=["2", "2-ragged", "2-and-4"])
def test_withheld_sums_time_out_and_the_gpu_stays_usable(g, H, dtype, exchange):
    """One CTA of every cluster waits in one exchange for an arrival that never comes
    and gives up, and its peers after it: every wait ends at its limit, the call records the timeout, and the same calls without
    the hook give what they gave before."""
    rows = 1200
    x, gen = inputs(H, rows, H, dtype, True, "channel", True, True)
    dz = torch.randn(rows, H, generator=gen).to(dtype).cuda()
    y, h = dev(x["y"]), dev(x["h"])
    kw = dict(post_weight=dev(x["post_w"]), gate=dev(x["gate"]), scale=0.5, pre_weight=dev(x["pre_w"]), eps=EPS)
    calls = [lambda: g.norm_residual(y, h, **kw), lambda: g.norm_residual_backward(dz, None, h, y, **kw)]
    for run in calls:
        want = run()
        assert g.device_error(clear=True) == 0
        g.testing_withhold_sum(exchange, wait_limit_us=2000)
        try:
            run()
            torch.cuda.synchronize()    # raises if the kernel faulted
        finally:
            g.testing_withhold_sum(None)
        assert g.device_error(clear=True) == g.DEVERR_TIMEOUT
        assert all(torch.equal(a, b) for a, b in zip(want, run()))
        assert g.device_error() == 0
