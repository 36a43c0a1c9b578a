"""spec_cross_entropy's gradients write nothing behind their outputs and their
workspace, with every row in use, and the bias gradient is right where the last
tile of rows is mostly empty."""
import pytest
import torch

import draft_verification_row_amd as sv
from test_gpu_cross_entropy import check, make
from test_gpu_embedding import DT, U, at_offset, close

pytestmark = pytest.mark.gpu

# rows that leave a tile of 64 a wave without any; K of whole and of broken chunks
CASES = [(1, 700, 64), (6, 5025, 777), (16, 3200, 1024), (32, 1000, 31), (65, 130, 130), (77, 1000, 64), (77, 3201, 515),
         (80, 16000, 768), (129, 700, 72), (130, 8192, 1024), (200, 4096, 512)]


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,K", CASES)
def test_gradients_stay_in_their_workspace(M, V, K, dtype, off):
    """off: of the weight from 16 bytes, in elements."""
    lib = sv.load_library()
    st = torch.cuda.current_stream().cuda_stream
    dt, code = DT[dtype], int(dtype == "bf16")
    (x, w, b), tok, gl, ge = make(M, V, K, dt, True, 0, 0.0, 1)
    w = at_offset(w, off)
    guard = 2 * V + 512  # elements
    f = lambda n, t: torch.full((n + guard,), 7, dtype=t, device="cuda")  # noqa: E731
    loss, lse, stats = (torch.empty(n, device="cuda") for n in (M, M, 2 * M))
    status = torch.empty(M, dtype=torch.int32, device="cuda")
    grads, sizes = [f(n, dt) for n in (M * K, V * K, V)], (M * K, V * K, V)
    n1 = lib.spec_cross_entropy_workspace_bytes(code, M, V, K)
    n2 = lib.spec_cross_entropy_grad_workspace_bytes(code, M, V, K)
    w1, w2 = (torch.full((n + 4 * guard,), 3, dtype=torch.uint8, device="cuda") for n in (n1, n2))
    assert lib.spec_cross_entropy(x.data_ptr(), w.data_ptr(), b.data_ptr(), code, tok.data_ptr(), M, V, K, loss.data_ptr(),
                                  lse.data_ptr(), status.data_ptr(), stats.data_ptr(), w1.data_ptr(), n1, st) == 0
    assert lib.spec_cross_entropy_grad(x.data_ptr(), w.data_ptr(), b.data_ptr(), code, tok.data_ptr(), stats.data_ptr(),
                                       gl.data_ptr(), ge.data_ptr(), M, V, K, *(g.data_ptr() for g in grads), w2.data_ptr(), n2, st) == 0
    torch.cuda.synchronize()
    assert (w1[n1:] == 3).all() and (w2[n2:] == 3).all()
    for g, n in zip(grads, sizes):
        assert (g[n:] == 7).all()


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,K", CASES)
def test_gradients_with_every_row_in_use(M, V, K, dtype, off):
    check(M, V, K, dtype, bias=True, pad=0.0, off=off)


def test_more_tiles_than_a_launch_counts():
    """2^24 tiles of 64 x 64, whose threads pass 32 bits: they go in two launches.
    Four different rows of x, so that the float64 form is small.  Tolerances as in
    test_gpu_cross_entropy: a row's 4096 parts are joined 256 to a thread, after
    18 values in a lane and before 4 more steps."""
    M = V = 1 << 18
    K, last = 8, (1 << 18) - 64
    g = torch.Generator(device="cuda").manual_seed(1)
    w = at_offset((torch.randn(V, K, generator=g, device="cuda") / 2).bfloat16(), 1)
    b = (torch.randn(V, generator=g, device="cuda") / 2).bfloat16()
    rows = torch.randn(4, K, generator=g, device="cuda").bfloat16()
    x = rows.repeat(M // 4, 1)
    tok = torch.randint(-1, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    tok[:128] = torch.arange(last - 64, V, dtype=torch.int32, device="cuda")  # on either side
    out = sv.spec_cross_entropy(x, w, tok, b)
    rd, wd, bd = rows.double(), w.double(), b.double()
    z = rd @ wd.t() + bd
    e = (2 * U * (K + 9) * (rd.abs() @ wd.abs().t() + bd.abs())).amax(1).repeat(M // 4)
    n = torch.logsumexp(z, 1)
    on = tok >= 0
    loss = n.repeat(M // 4) - z[torch.arange(M, device="cuda") % 4, tok.long().clamp_min(0)]
    lse = n.repeat(M // 4)
    size = U * (600 + 4 * lse.abs() + 4 * loss.abs())
    close(out.lse[on], lse[on], (e + size)[on], "lse")
    close(out.loss[on], loss[on], (2 * e + size)[on], "loss")
    assert (out.loss[~on] == 0).all() and (out.lse[~on] == 0).all() and (out.status == 0).all()
