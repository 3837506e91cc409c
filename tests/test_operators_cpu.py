"""Refusals of the MoE block's operators on a machine without a GPU: the C ABI's
host checks (fake device addresses, every call returns before any CUDA call)
and the Python binding's checks (stand-in tensors)."""
import ctypes as C

import pytest
import torch

from .test_binding_cpu import FakeCudaTensor

P = 0x7f0000000000
S = None


@pytest.fixture(scope="module")
def gemm():
    from fp8_block_scaled_x128_b200 import gemm
    return gemm


OK, INVALID, MISALIGNED = 0, 1, 2


def call(lib, name, good, **changed):
    """The entry point's status with some of its good arguments changed."""
    assert set(changed) <= set(good)
    return getattr(lib, name)(*dict(good, **changed).values(), S)


MASKED = dict(x=P, dt=0, T=4, K=256, expert=P, topk=2, G=8, Mmax=64, A=P, sa=P, ld=64, pos=P, masked_m=P)


@pytest.mark.parametrize("status,changed", [
    (INVALID, dict(dt=2)), (INVALID, dict(T=-1)), (INVALID, dict(K=0)), (INVALID, dict(K=200)),
    (INVALID, dict(K=65536 + 128)), (INVALID, dict(topk=0)), (INVALID, dict(topk=17)), (INVALID, dict(G=0)),
    (INVALID, dict(G=257)), (INVALID, dict(Mmax=0)), (INVALID, dict(ld=60)), (MISALIGNED, dict(ld=66)),
    (INVALID, dict(T=1 << 30, topk=4)), (INVALID, dict(G=256, Mmax=1 << 23, ld=1 << 23)),
    (INVALID, dict(x=None)), (INVALID, dict(expert=None)), (INVALID, dict(A=None)), (INVALID, dict(sa=None)),
    (INVALID, dict(pos=None)), (INVALID, dict(masked_m=None)), (MISALIGNED, dict(x=P + 8)),
    (MISALIGNED, dict(A=P + 8)), (MISALIGNED, dict(sa=P + 4)), (MISALIGNED, dict(expert=P + 2)),
    (MISALIGNED, dict(pos=P + 1)), (MISALIGNED, dict(masked_m=P + 2))])
def test_dispatch_masked_refuses(gemm, status, changed):
    assert call(gemm.lib, "fp8g_moe_dispatch_masked", MASKED, **changed) == status


PERMUTE = dict(x=P, dt=0, T=4, N=64, expert=P, topk=2, G=8, blocks=9, xs=P, pos=P, mi=P)


@pytest.mark.parametrize("status,changed", [
    (INVALID, dict(dt=-1)), (INVALID, dict(T=-1)), (INVALID, dict(N=0)), (MISALIGNED, dict(N=60)),
    (INVALID, dict(N=(1 << 20) + 8)),
    (INVALID, dict(topk=0)), (INVALID, dict(topk=17)), (INVALID, dict(G=0)), (INVALID, dict(G=257)),
    (INVALID, dict(blocks=8)), (INVALID, dict(blocks=1 << 24)), (INVALID, dict(T=1 << 30, topk=4, blocks=1 << 23)),
    (INVALID, dict(x=None)), (INVALID, dict(expert=None)), (INVALID, dict(xs=None)), (INVALID, dict(pos=None)),
    (INVALID, dict(mi=None)), (INVALID, dict(T=0, mi=None)), (MISALIGNED, dict(x=P + 2)), (MISALIGNED, dict(xs=P + 8)),
    (MISALIGNED, dict(expert=P + 2)), (MISALIGNED, dict(pos=P + 2)), (MISALIGNED, dict(mi=P + 2))])
def test_permute_refuses(gemm, status, changed):
    assert call(gemm.lib, "fp8g_moe_permute", PERMUTE, **changed) == status


PERMUTE_BWD = dict(dxs=P, dt=1, blocks=9, N=64, pos=P, T=4, topk=2, dx=P)


@pytest.mark.parametrize("status,changed", [
    (INVALID, dict(dt=2)), (INVALID, dict(blocks=-1)), (INVALID, dict(blocks=1 << 24)), (INVALID, dict(N=0)),
    (MISALIGNED, dict(N=12)), (INVALID, dict(T=-1)), (INVALID, dict(topk=17)), (INVALID, dict(dxs=None)),
    (INVALID, dict(pos=None)), (INVALID, dict(dx=None)), (MISALIGNED, dict(dxs=P + 8)), (MISALIGNED, dict(dx=P + 4)),
    (MISALIGNED, dict(pos=P + 2)), (OK, dict(T=0, dxs=None, pos=None, dx=None))])
def test_permute_backward_refuses(gemm, status, changed):
    assert call(gemm.lib, "fp8g_moe_permute_backward", PERMUTE_BWD, **changed) == status


COMBINE_BWD = dict(dout=P, D=P, N=256, pos=P, w=P, T=4, topk=2, blocks=9, dD=None, q=P, sa=P, ld=1152, dw=P)


@pytest.mark.parametrize("status,changed", [
    (INVALID, dict(N=0)), (INVALID, dict(N=200)), (MISALIGNED, dict(N=196, q=None, dD=P)), (INVALID, dict(T=-2)),
    (INVALID, dict(topk=0)), (INVALID, dict(topk=17)), (INVALID, dict(blocks=-1)), (INVALID, dict(blocks=1 << 24)),
    (INVALID, dict(ld=1148)), (MISALIGNED, dict(ld=1154)), (INVALID, dict(dD=P)), (INVALID, dict(q=None)),
    (INVALID, dict(sa=None)), (INVALID, dict(D=None)), (INVALID, dict(dout=None)), (INVALID, dict(pos=None)),
    (MISALIGNED, dict(dout=P + 8)), (MISALIGNED, dict(D=P + 8)), (MISALIGNED, dict(q=P + 8)),
    (MISALIGNED, dict(q=None, dD=P + 2)), (MISALIGNED, dict(sa=P + 4)), (MISALIGNED, dict(w=P + 2)),
    (MISALIGNED, dict(dw=P + 2)), (MISALIGNED, dict(pos=P + 3)), (OK, dict(T=0, dout=None, D=None, pos=None))])
def test_combine_backward_refuses(gemm, status, changed):
    assert call(gemm.lib, "fp8g_moe_combine_backward", COMBINE_BWD, **changed) == status


NAN, INF = float("nan"), float("inf")
NORM = dict(y=P, h=P, dt=0, rows=4, H=256, post=P, gate=P, kind=1, scale=1.0, pre=P, eps=1e-6, h_out=P, z=P, q=None,
            sa=None, ld=0)
FP8 = dict(z=None, q=P, sa=P, ld=4)


@pytest.mark.parametrize("status,changed", [
    (INVALID, dict(dt=2)), (INVALID, dict(rows=-1)), (INVALID, dict(H=0)), (INVALID, dict(H=16384 + 8)),
    (MISALIGNED, dict(H=252)), (INVALID, dict(kind=3)), (INVALID, dict(kind=-1)), (INVALID, dict(kind=0)),
    (INVALID, dict(gate=None)), (INVALID, dict(scale=NAN)), (INVALID, dict(scale=INF)), (INVALID, dict(eps=0.0)),
    (INVALID, dict(eps=-1e-6)), (INVALID, dict(eps=NAN)), (INVALID, dict(eps=INF)), (INVALID, dict(z=None)),
    (INVALID, dict(q=P, sa=P, ld=4)), (INVALID, dict(FP8, H=264)), (INVALID, dict(FP8, ld=0)), (INVALID, dict(FP8, sa=None)),
    (INVALID, dict(FP8, rows=5)), (MISALIGNED, dict(FP8, ld=6)), (INVALID, dict(y=None)), (INVALID, dict(h_out=None)),
    (MISALIGNED, dict(y=P + 8)), (MISALIGNED, dict(h=P + 8)), (MISALIGNED, dict(h_out=P + 8)), (MISALIGNED, dict(z=P + 8)),
    (MISALIGNED, dict(FP8, q=P + 8)), (MISALIGNED, dict(FP8, sa=P + 4)), (MISALIGNED, dict(post=P + 4)),
    (MISALIGNED, dict(pre=P + 8)), (MISALIGNED, dict(gate=P + 4)), (MISALIGNED, dict(gate=P + 2, kind=2)),
    (OK, dict(rows=0, y=None, h_out=None, z=None))])
def test_norm_refuses(gemm, status, changed):
    assert call(gemm.lib, "fp8g_norm_residual", NORM, **changed) == status


NORM_BWD = dict(dz=P, dh_out=P, h_out=P, y=P, dt=1, rows=4, H=256, post=P, gate=P, kind=1, scale=1.0, pre=P, eps=1e-6,
                dh=P, dy=P, dpre=P, dpost=P, dgate=P, ws=P, ws_bytes=1 << 20)


@pytest.mark.parametrize("status,changed", [
    (INVALID, dict(dt=5)), (INVALID, dict(rows=-1)), (INVALID, dict(H=0)), (INVALID, dict(H=16392)),
    (MISALIGNED, dict(H=36)), (INVALID, dict(kind=0)), (INVALID, dict(gate=None, kind=0)), (INVALID, dict(post=None)),
    (INVALID, dict(eps=0.0)), (INVALID, dict(scale=INF)), (INVALID, dict(ws=None)), (INVALID, dict(ws_bytes=4 * 256 * 4)),
    (INVALID, dict(dz=None, dh_out=None)), (INVALID, dict(h_out=None)), (INVALID, dict(y=None)), (INVALID, dict(dh=None)),
    (INVALID, dict(dy=None)), (MISALIGNED, dict(dz=P + 8)), (MISALIGNED, dict(dh_out=P + 8)), (MISALIGNED, dict(h_out=P + 8)),
    (MISALIGNED, dict(y=P + 8)), (MISALIGNED, dict(dh=P + 8)), (MISALIGNED, dict(dy=P + 8)), (MISALIGNED, dict(ws=P + 8)),
    (MISALIGNED, dict(dpre=P + 2)), (MISALIGNED, dict(dpost=P + 2)), (MISALIGNED, dict(dgate=P + 2)),
    (MISALIGNED, dict(gate=P + 8)),
    (OK, dict(rows=0, dz=None, dh_out=None, h_out=None, y=None, dh=None, dy=None, dpre=None, dpost=None, dgate=None))])
def test_norm_backward_refuses(gemm, status, changed):
    assert call(gemm.lib, "fp8g_norm_residual_backward", NORM_BWD, **changed) == status


def test_workspace_sizes(gemm):
    f = gemm.lib.fp8g_norm_residual_backward_workspace_bytes
    assert f(-1, 256) == f(4, 0) == f(4, 16392) == f(4, 12) == 0
    assert f(4, 256) >= 2 * 4 * 256 * 4
    assert f(1 << 30, 16384) < 1 << 28      # bounded by the GPU, not by the rows


@pytest.mark.parametrize("H", [8, 128, 520, 1024, 2048, 2112, 4096, 7168, 8200, 12416, 16384])
def test_a_workspace_for_the_largest_batch_serves_every_smaller_one(gemm, H):
    """A caller keeps one workspace for its largest batch: the size never falls
    as the rows grow, past the row counts where the rows of a CTA go up by one
    (multiples of 148 and of what a smaller grid has) too."""
    f = gemm.lib.fp8g_norm_residual_backward_workspace_bytes
    sizes = [f(r, H) for r in range(0, 12000)] + [f(r, H) for r in (1 << 14, 148 * 997, 1 << 20, 1 << 30, 2 ** 31 - 1)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
@pytest.mark.parametrize("name,good", [("fp8g_moe_dispatch_masked", MASKED), ("fp8g_moe_permute", PERMUTE),
                                       ("fp8g_moe_permute_backward", PERMUTE_BWD),
                                       ("fp8g_moe_combine_backward", COMBINE_BWD), ("fp8g_norm_residual", NORM),
                                       ("fp8g_norm_residual_backward", NORM_BWD)])
def test_good_arguments_reach_the_device(gemm, name, good):
    assert call(gemm.lib, name, good) == 4       # FP8G_ERR_CUDA: there is no GPU here


# ---------------------------------------------------------------- the binding
def fake(shape, dtype=torch.bfloat16, index=0):
    t = FakeCudaTensor(shape, dtype, index)
    t.dim = lambda: len(shape)
    t.get_device = lambda: index
    return t


I32, F32, U8 = torch.int32, torch.float32, torch.uint8


def test_binding_refuses_wrong_shapes_and_types(gemm):
    x, e, pos = fake((4, 256)), fake((8,), I32), fake((8,), I32)
    with pytest.raises(TypeError, match="expert"):
        gemm.moe_dispatch_masked(x, fake((9,), I32), 2, 4, 64)
    with pytest.raises(TypeError, match="expert"):
        gemm.moe_permute(x, fake((8,), torch.int64), 2, 4)
    with pytest.raises(TypeError, match="x"):
        gemm.moe_permute(fake((4, 256), torch.float16), e, 2, 4)
    with pytest.raises(TypeError, match="x"):
        gemm.moe_dispatch_masked(fake((2, 2, 256)), e, 2, 4, 64)
    with pytest.raises(ValueError, match="128-row"):
        gemm.moe_permute_backward(fake((100, 64)), pos, 4, 2)
    with pytest.raises(TypeError, match="pos"):
        gemm.moe_permute_backward(fake((128, 64)), pos, 5, 2)
    with pytest.raises(TypeError, match="dout"):
        gemm.moe_combine_backward(fake((4, 256), F32), fake((128, 256)), pos, None, 4, 2)
    with pytest.raises(TypeError, match="w"):
        gemm.moe_combine_backward(x, fake((128, 256)), pos, fake((4, 2), F32), 4, 2)
    with pytest.raises(TypeError, match="h"):
        gemm.norm_residual(x, fake((4, 256), F32))
    with pytest.raises(TypeError, match="gate"):
        gemm.norm_residual(x, gate=fake((4,), F32))
    with pytest.raises(TypeError, match="gate"):
        gemm.norm_residual(x, gate=fake((256, 1), F32))
    with pytest.raises(TypeError, match="post_weight"):
        gemm.norm_residual(x, post_weight=fake((256,), torch.bfloat16))
    with pytest.raises(TypeError, match="dz"):
        gemm.norm_residual_backward(fake((4, 128)), None, x, x)
    t = fake((4, 256))
    t.is_contiguous = lambda: False
    with pytest.raises(TypeError, match="y"):
        gemm.norm_residual(t)


def test_binding_refuses_operands_on_two_devices(gemm):
    x, e = fake((4, 256)), fake((8,), I32)
    with pytest.raises(ValueError, match="one device"):
        gemm.moe_permute(x, fake((8,), I32, 1), 2, 4)
    with pytest.raises(ValueError, match="one device"):
        gemm.moe_dispatch_masked(x, fake((8,), I32, 1), 2, 4, 64)
    with pytest.raises(ValueError, match="one device"):
        gemm.moe_permute_backward(fake((128, 64)), fake((8,), I32, 1), 4, 2)
    with pytest.raises(ValueError, match="one device"):
        gemm.moe_combine_backward(x, fake((128, 256), index=1), e, None, 4, 2)
    with pytest.raises(ValueError, match="one device"):
        gemm.norm_residual(x, fake((4, 256), index=1))
    with pytest.raises(ValueError, match="one device"):
        gemm.norm_residual_backward(x, None, x, fake((4, 256), index=2))


class OtherStream:
    """On another device than the operands: refused behind the operands' checks."""
    device = torch.device("cuda", 1)


def test_binding_takes_slots_of_any_shape(gemm):
    """A router's [T, topk] experts, and positions kept in that shape, as the
    quantised dispatch and the combine take them."""
    x, e = fake((4, 256)), fake((4, 2), I32)
    for call_it in (lambda: gemm.moe_permute(x, e, 2, 4, stream=OtherStream),
                    lambda: gemm.moe_dispatch_masked(x, e, 2, 4, 64, stream=OtherStream),
                    lambda: gemm.moe_permute_backward(fake((128, 64)), e, 4, 2, stream=OtherStream),
                    lambda: gemm.moe_combine_backward(x, fake((128, 256)), e, None, 4, 2, stream=OtherStream)):
        with pytest.raises(ValueError, match="stream is on"):
            call_it()
    for bad in (fake((4, 3), I32), fake((4, 2), torch.int64), fake((2, 4, 2), I32)):
        with pytest.raises(TypeError, match="expert"):
            gemm.moe_permute(x, bad, 2, 4)
        with pytest.raises(TypeError, match="expert"):
            gemm.moe_dispatch_masked(x, bad, 2, 4, 64)
        with pytest.raises(TypeError, match="pos"):
            gemm.moe_permute_backward(fake((128, 64)), bad, 4, 2)
        with pytest.raises(TypeError, match="pos"):
            gemm.moe_combine_backward(x, fake((128, 256)), bad, None, 4, 2)


def test_withheld_sum_hook_checks_its_arguments(gemm):
    f = gemm.lib.fp8g_testing_withhold_sum
    assert f(1, 50) == f(1, 2_000_000) == INVALID     # limits below 100 us and above 1 s
    assert f(2, 2000) == INVALID                      # an exchange that the hook does not reach
    assert f(1, 2000) == OK and f(-1, 0) == OK        # on, and off again
