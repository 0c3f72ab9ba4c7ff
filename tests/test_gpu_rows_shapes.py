"""The few-row operators at the shapes where their work is cut differently: rows of more than 8192 channels (several parts
a row in the preparation, which finds the row's largest value in a second read), several pieces of them a CTA, more
clusters of one launch than fit at once, rows that lie more than 2^32 elements apart, calls joined within one capture."""
import pytest
import torch

from rows_case import Weight, assert_within, check_norm, norm_reference, rows_input, rows_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    import video_diffusion_w4a4_b200 as m
    return m


_weights = {}


def weight(dq, Ci, Co, rank):
    if (Ci, Co, rank) not in _weights:
        w = Weight(dq, Ci, Co, rank, seed=Ci, bias=True)
        _weights[Ci, Co, rank] = (w, w.device())
    return _weights[Ci, Co, rank]


def product(dq, dev, w, x, sc, fmt, rows, gelu=False, stream=None, calls=1):
    y = torch.full((rows + 1, w.Co), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((dq.dq_rows_workspace_bytes(rows, w.Ci, w.Co, w.rank),), 0xFF, dtype=torch.uint8, device="cuda")
    xd, sd = x.cuda(), sc.cuda() if sc is not None else None
    for _ in range(calls):
        dq.dq_rows_forward(xd, rows, w.Ci, w.Co, w.rank, *dev, y, ws, ws.numel(), x_format=fmt, x_scales=sd,
                           epilogue=dq.DQ_EPILOGUE_GELU if gelu else dq.DQ_EPILOGUE_NONE, stream=stream)
    torch.cuda.synchronize()
    assert dq.dq_read_device_status(ws) == 0 and (y[rows:] == -7).all()
    return y[:rows].cpu()


def hard_rows(rows, Ci, fmt, seed):
    """Rows whose largest value is their last channel's, one of zeros, one that is zero past the first 8192 channels,
    and (returned apart) rows with a NaN or an infinity in their last part."""
    v, x, sc = rows_input(rows, Ci, fmt, seed=seed)
    v, code = v.clone(), x if fmt == 0 else x.view(torch.uint8)
    bad = []
    if rows > 2:
        code[1] = 0
        v[1] = 0
        code[2, 8192:] = 0
        v[2, 8192:] = 0
    for m in range(0, rows, 5):
        if m not in (1, 2):
            x[m, Ci - 1] = 440.0 if fmt else float(v[m].abs().max() * 2)
            v[m, Ci - 1] = x[m, Ci - 1].double() * (sc[m, -1].double() if fmt else 1.0)
    if rows > 3:
        bad.append(3)
        x[3, Ci - 2] = float("nan")
    if rows > 8:
        bad.append(8)
        if fmt == 0:
            x[8, Ci - 1] = float("-inf")
        else:
            sc[8, -1] = float("inf")
    return v, x, sc, bad


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("Ci,Co,rank,rows", [(13824, 512, 32, 1), (13824, 512, 32, 4), (13824, 512, 32, 9), (13824, 512, 32, 33),
                                             (13824, 512, 32, 130), (16640, 256, 16, 3), (16640, 256, 16, 8),
                                             (16640, 256, 16, 35), (8448, 256, 48, 700)])
def test_rows_of_several_parts(dq, Ci, Co, rank, rows, fmt):
    w, dev = weight(dq, Ci, Co, rank)
    v, x, sc, bad = hard_rows(rows, Ci, fmt, seed=rows + fmt)
    gelu = rows % 2 == 1
    y = product(dq, dev, w, x, sc, fmt, rows, gelu, calls=2)
    assert torch.isnan(y[bad].float()).all()
    fine = [m for m in range(rows) if m not in bad]
    ref, tol = rows_reference(w, v[fine], gelu)
    assert_within(y[fine], ref, tol, "Y")


@pytest.mark.parametrize("rows", [1, 3, 8])
def test_one_launch_with_more_clusters_than_fit_at_once(dq, rows):
    w, dev = weight(dq, 256, 20480, 16)
    for fmt in (0, 1, 2):
        v, x, sc = rows_input(rows, 256, fmt, seed=rows + fmt)
        ref, tol = rows_reference(w, v, fmt == 1)
        assert_within(product(dq, dev, w, x, sc, fmt, rows, fmt == 1, calls=3), ref, tol, "Y")


@pytest.mark.parametrize("fmt", [0, 2])
def test_rows_far_apart(dq, fmt):
    """Strides that take the third row past 2^32 elements."""
    C, rows, stride = 512, 3, (1 << 31) + 64
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    w, dev = weight(dq, C, 768, 32)
    v, x, sc = rows_input(rows, C, fmt, seed=1)
    xbuf = torch.empty(2 * stride + C, dtype=x.dtype, device="cuda").as_strided((rows, C), (stride, 1))
    ybuf = torch.empty(2 * stride + 768, dtype=torch.bfloat16, device="cuda").as_strided((rows, 768), (stride, 1))
    xbuf.copy_(x)
    ws = torch.full((dq.dq_rows_workspace_bytes(rows, C, 768, 32),), 0xFF, dtype=torch.uint8, device="cuda")
    dq.dq_rows_forward(xbuf, rows, C, 768, 32, *dev, ybuf, ws, ws.numel(), x_stride=stride, x_format=fmt,
                       x_scales=sc.cuda() if fmt else None, y_stride=stride)
    torch.cuda.synchronize()
    ref, tol = rows_reference(w, v, False)
    assert_within(ybuf.cpu(), ref, tol, "Y")
    if fmt == 0:   # the norm of the same rows, written where the product's Y was
        r = torch.randn(rows, C, generator=torch.Generator().manual_seed(2)).bfloat16()
        for shift in (0, 1):   # wide and element accesses
            yv = ybuf.as_strided((rows, C), (stride, 1), shift)
            dq.dq_rmsnorm_forward(xbuf, rows, C, yv, x_stride=stride, residual=r.cuda(), y_stride=stride)
            torch.cuda.synchronize()
            h, y = norm_reference(x, r, None, 1e-6)
            check_norm(dq, h, y, C, 0, None, yv.cpu(), None)
        del yv
    del xbuf, ybuf
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [2, 30])
def test_not_finite_rows_pass_through_gelu(dq, rows):
    w, dev = weight(dq, 512, 768, 32)
    v, x, _ = rows_input(rows, 512, 0, seed=3)
    x[1, 5] = float("nan")
    y = product(dq, dev, w, x, None, 0, rows, gelu=True)
    assert torch.isnan(y[1].float()).all()
    fine = [m for m in range(rows) if m != 1]
    ref, tol = rows_reference(w, v[fine], True)
    assert_within(y[fine], ref, tol, "Y")


@pytest.mark.parametrize("rows", [4, 30])
def test_two_branches_of_one_capture(dq, rows):
    """A norm whose rows two products on two streams read, and a norm of both products' outputs: the branches part and
    join within one captured graph, so a launch has more than one before it."""
    w, dev = weight(dq, 512, 512, 32)
    v, x, _ = rows_input(rows, 512, 0, seed=4)
    xd = x.cuda()
    n, a, b, z = (torch.zeros(rows, 512, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    wss = [torch.zeros(dq.dq_rows_workspace_bytes(rows, 512, 512, 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()

    def calls():
        dq.dq_rmsnorm_forward(xd, rows, 512, n, stream=s0)
        s1.wait_stream(s0)
        dq.dq_rows_forward(n, rows, 512, 512, 32, *dev, a, wss[0], wss[0].numel(), stream=s0)
        dq.dq_rows_forward(n, rows, 512, 512, 32, *dev, b, wss[1], wss[1].numel(), epilogue=dq.DQ_EPILOGUE_GELU, stream=s1)
        s0.wait_stream(s1)
        dq.dq_rmsnorm_forward(a, rows, 512, z, residual=b, stream=s0)

    torch.cuda.synchronize()
    calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in (n, a, b, z)]
    h, ref = norm_reference(want[1].cpu(), want[2].cpu(), None, 1e-6)
    check_norm(dq, h, ref, 512, 0, None, want[3].cpu(), None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s0):
        calls()
    for _ in range(3):
        for t in (n, a, b, z):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip((n, a, b, z), want))
    del graph


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_norm_with_the_largest_eps(dq, fmt):
    x = torch.ldexp(torch.randn(3, 320, generator=torch.Generator().manual_seed(1)), torch.tensor(62)).bfloat16()
    y = torch.empty(3, 320, dtype=torch.bfloat16 if fmt == 0 else torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(3, 1 if fmt == 1 else 5, device="cuda") if fmt else None
    eps = float(torch.finfo(torch.float32).max)
    dq.dq_rmsnorm_forward(x.cuda(), 3, 320, y, eps=eps, y_format=fmt, y_scales=sc)
    torch.cuda.synchronize()
    h, ref = norm_reference(x, None, None, eps)
    check_norm(dq, h, ref, 320, fmt, None, y.cpu(), sc.cpu() if fmt else None)
