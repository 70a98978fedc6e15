"""Outputs that meet inputs are refused; matrices that lie side by side in one
buffer do not meet."""
import ctypes

import pytest
import torch

import gemm_amax_reduce_amd as nv

_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer argument tests run only without a GPU")
SHAPE, HIP = -2, -4
A = 1 << 20


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def _meets(a, lda, b, ldb, rows, cols):
    """By the elements' addresses."""
    at = lambda p, ld: {p + 2 * (r * ld + c) + i for r in range(rows) for c in range(cols) for i in (0, 1)}
    return bool(at(a, lda) & at(b, ldb))


@_no_gpu
@pytest.mark.parametrize("rows", [1, 2, 3])
def test_distillation(L, rows):
    """Every shift of one matrix against another in the same rows; what does
    not meet gets as far as the launch, which fails without a GPU."""
    cols = 3
    for ld in (3, 5, 6, 8):
        for shift in range(-rows * ld - 2, rows * ld + 3):
            b = A + 2 * shift
            got = L.nvfp4_distill_topk_backward(A, 1, rows, cols, ld, None, 64, None, 1, 0, 1.0, 4 * A, 4 * A, b, ld,
                                                None)
            assert got == (SHAPE if _meets(A, ld, b, ld, rows, cols) else HIP), (ld, shift)


@pytest.mark.gpu
def test_distillation_beside_its_logits():
    """Logits and gradient as the two halves of one buffer."""
    buf = torch.full((6, 200), 7.0, device="cuda", dtype=torch.bfloat16)
    buf[:, :90] = torch.randn((6, 90), device="cuda")
    z, dz = buf[:, :90], buf[:, 100:190]
    idx = torch.randint(0, 90, (6, 4), device="cuda")
    t, weight = torch.randn((6, 4), device="cuda"), torch.rand(6, device="cuda")
    want = nv.nvfp4_distill_topk_step(z.clone(), idx, t, weight)
    got = nv.nvfp4_distill_topk_step(z, idx, t, weight, out=dz)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    assert torch.all(buf[:, 90:100] == 7) and torch.all(buf[:, 190:] == 7)


@_no_gpu
@pytest.mark.parametrize("xd,yd", [(1, 1), (0, 1), (1, 0)])
@pytest.mark.parametrize("rows", [1, 3])
def test_layer_norm(L, rows, xd, yd):
    """y against x, and the gradient dx (x's type) against dy (of type yd) and x."""
    cols, size = 3, {0: 4, 1: 2}
    far, ws = 4 * A, 8 * A
    for ldx, ldy in ((3, 3), (8, 8), (8, 16), (16, 8)):
        for shift in range(-4 * rows * 16, 4 * rows * 16 + 1, 4):
            at = lambda p, ld, d: {p + size[d] * (r * ld + c) + i for r in range(rows) for c in range(cols)
                                   for i in range(size[d])}
            b = A + shift
            fwd = L.nvfp4_layer_norm(A, xd, rows, cols, ldx, None, None, 0, 1e-5, b, yd, ldy, far, far, None, None, 0,
                                     None)
            # dx first against dy, then against x
            back_dy = L.nvfp4_layer_norm_backward(b, yd, ldy, far, xd, rows, cols, cols, far, far, None, 0, A, ldx,
                                                  None, None, 0, ws, 1 << 30, None)
            back_x = L.nvfp4_layer_norm_backward(far, xd, cols, b, xd, rows, cols, ldy, far, far, None, 0, A, ldx, None,
                                                 None, 0, ws, 1 << 30, None)
            for got, d in ((fwd, yd), (back_dy, yd), (back_x, xd)):
                meets = bool(at(A, ldx, xd) & at(b, ldy, d))
                if meets or ldx * size[xd] == ldy * size[d]:
                    assert got == (SHAPE if meets else HIP), (ldx, ldy, shift)
                else:                            # of two pitches: refused where the whole ranges meet
                    assert got in (SHAPE, HIP)


@pytest.mark.gpu
def test_layer_norm_refuses_its_input():
    x = torch.randn((6, 64), device="cuda")
    for out in (x, x.view(12, 32)[:6].view(3, 64)):
        with pytest.raises(nv.NVFP4Error, match="shape"):
            nv.nvfp4_layer_norm(x[:out.shape[0]], out=out)
    buf = torch.full((6, 200), 7.0, device="cuda")
    buf[:, :90] = torch.randn((6, 90), device="cuda")
    want = nv.nvfp4_layer_norm(buf[:, :90].clone())[0]
    assert torch.equal(nv.nvfp4_layer_norm(buf[:, :90], out=buf[:, 100:190])[0], want)
    assert torch.all(buf[:, 90:100] == 7) and torch.all(buf[:, 190:] == 7)


@_no_gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("tokens", [1, 3])
def test_matvec(L, mx, tokens):
    """y (f32, N = 5) against x (bf16, K = 32)."""
    n, k, far = 5, 32, 4 * A
    w = nv._MXTensor(far, far, n, k) if mx else nv._CTensor(far, far, far, n, k)
    fn = L.mxfp4_matvec if mx else L.nvfp4_matvec
    for ldx, ldy in ((32, 16), (48, 24), (64, 32)):
        at = lambda p, ld, size, cols: {p + size * r * ld + i for r in range(tokens) for i in range(size * cols)}
        for shift in range(-256, 257, 4):
            y = A + shift
            meets = bool(at(A, ldx, 2, k) & at(y, ldy, 4, n))
            got = fn(ctypes.byref(w), A, 1, tokens, ldx, y, 0, ldy, None, 0, None)
            assert got == (SHAPE if meets else HIP), (ldx, shift)


@pytest.mark.gpu
def test_matvec_refuses_its_input():
    x = torch.randn((4, 64), device="cuda")
    w = nv.nvfp4_quantize(torch.randn((64, 64), device="cuda"))
    with pytest.raises(nv.NVFP4Error, match="shape"):
        nv.nvfp4_matvec(w, x, out=x)
    buf = torch.cat([x, torch.zeros_like(x)], 1)
    want = nv.nvfp4_matvec(w, x)
    assert torch.equal(nv.nvfp4_matvec(w, buf[:, :64], out=buf[:, 64:]), want) and torch.equal(buf[:, :64], x)
