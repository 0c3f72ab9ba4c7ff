"""The few-row operators on the GPU against their definitions in 64 bits (rows_case.py has the bounds)."""
import numpy as np
import pytest
import torch

from rows_case import (Weight, assert_within, bf16, check_norm, norm_reference, quantise_rows, rows_input,
                       rows_reference)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    import video_diffusion_w4a4_b200 as m
    return m


_weights = {}


def weight(dq, Ci, Co, rank, **kw):
    key = (Ci, Co, rank, tuple(sorted(kw.items())))
    if key not in _weights:
        w = Weight(dq, Ci, Co, rank, **kw)
        _weights[key] = (w, w.device())
    return _weights[key]


# ------------------------------------------------------------------ RMS norm

SENTINEL = -7.0


def run_norm(dq, x, residual, gamma, fmt, eps=1e-6, pad=0, want_sum=True, extra_rows=2, shift=0, stream=None):
    """The call on device copies with `pad` columns and `extra_rows` rows around it, which must stay as they were."""
    rows, C = x.shape

    def strided(t, dtype):
        buf = torch.full((rows + extra_rows, C + pad + shift), SENTINEL, device="cuda").to(dtype)
        view = buf[:rows, shift:shift + C]
        if t is not None:
            view.copy_(t)
        return buf, view

    xb, xv = strided(x, torch.bfloat16)
    rb, rv = strided(residual, torch.bfloat16) if residual is not None else (None, None)
    sb, sv = strided(None, torch.bfloat16) if want_sum else (None, None)
    yb, yv = strided(None, torch.bfloat16 if fmt == 0 else torch.float8_e4m3fn)
    groups = 1 if fmt == 1 else -(-C // 64)
    sc = torch.full((rows + extra_rows, groups), SENTINEL, device="cuda") if fmt else None
    g = gamma.cuda() if gamma is not None else None
    torch.cuda.synchronize()
    dq.dq_rmsnorm_forward(xv, rows, C, yv, x_stride=xv.stride(0), residual=rv,
                          residual_stride=rv.stride(0) if rv is not None else 0, sum_out=sv,
                          sum_stride=sv.stride(0) if sv is not None else 0, gamma=g, eps=eps, y_format=fmt,
                          y_stride=yv.stride(0), y_scales=sc, stream=stream)
    torch.cuda.synchronize()
    for buf in (sb, yb):
        if buf is not None:
            f = buf.float()
            assert (f[rows:] == SENTINEL).all() and (f[:, :shift] == SENTINEL).all() and (f[:, shift + C:] == SENTINEL).all()
    if sc is not None:
        assert (sc[rows:] == SENTINEL).all()
    assert torch.equal(xb[:rows, shift:shift + C].cpu().view(torch.int16), x.view(torch.int16))   # X as it was, NaN too
    return (sv.cpu() if sv is not None else None), yv.cpu(), (sc[:rows].cpu() if sc is not None else None)


def norm_input(rows, C, residual, gamma, seed=0):
    rng = np.random.default_rng(seed)
    t = lambda a: bf16(torch.from_numpy(a))  # noqa: E731
    x = rng.standard_normal((rows, C))
    r = rng.standard_normal((rows, C)) * np.exp(0.5 * rng.standard_normal(C))
    r[:, rng.integers(0, C, max(1, C // 100))] *= 50
    return t(x), t(r) if residual else None, t(1 + 0.2 * rng.standard_normal(C)) if gamma else None


NORM_SHAPES = [(1, 1), (3, 2), (5, 7), (2, 64), (2, 65), (33, 128), (1, 255), (4, 1337), (3, 2048), (1, 5120),
               (37, 5120), (2, 8191), (3, 13824), (1, 16384), (2, 32768), (1, 32767)]


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("rows,C", NORM_SHAPES)
def test_norm(dq, rows, C, fmt):
    for i, (residual, gamma, pad, shift) in enumerate([(True, True, 0, 0), (False, True, 1, 0), (True, False, 24, 8),
                                                       (False, False, 3, 1)]):
        x, r, g = norm_input(rows, C, residual, gamma, seed=C + i)
        s, y, sc = run_norm(dq, x, r, g, fmt, pad=pad, shift=shift, want_sum=i != 1)
        h, ref = norm_reference(x, r, g, 1e-6)
        check_norm(dq, h, ref, C, fmt, s, y, sc, f"norm {i}")


def test_norm_many_rows(dq):
    x, r, g = norm_input(5003, 640, True, True)
    for fmt in (0, 1, 2):
        s, y, sc = run_norm(dq, x, r, g, fmt)
        h, ref = norm_reference(x, r, g, 1e-6)
        check_norm(dq, h, ref, 640, fmt, s, y, sc)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("C", [200, 512])
def test_norm_of_hard_rows(dq, C, fmt):
    """Rows of zeros, of the largest and smallest magnitudes, one channel only, and x = -residual."""
    x, r, g = norm_input(8, C, True, True, seed=5)
    x[0], r[0] = 0, 0
    x[1], r[1] = 2.0 ** 60, 0
    x[2], r[2] = -2.0 ** -70, 0
    x[3], r[3] = 0, 0
    x[3, C - 1] = 3.0
    r[4] = -x[4]
    x[5], r[5] = 1.0, 2.0 ** -9
    g[7] = 0
    for eps in (1e-6, 0.0 if C == 200 else 1.0):
        if eps == 0.0:
            x[0, 0], x[4, 1] = 1.0, 0.5    # 0 / 0 is not asked for
        h, ref = norm_reference(x, r, g, eps)
        s, y, sc = run_norm(dq, x, r, g, fmt, eps=eps)
        check_norm(dq, h, ref, C, fmt, s, y, sc)
        if fmt and eps:
            assert (y[0].float() == 0).all() and (sc[0] == 0).all()


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_norm_not_finite_rows_stay_alone(dq, fmt):
    x, r, g = norm_input(6, 320, True, True, seed=9)
    x[1, 3], x[2, 319], r[4, 100] = float("nan"), float("inf"), float("-inf")
    h, ref = norm_reference(x, r, g, 1e-6)
    s, y, sc = run_norm(dq, x, r, g, fmt)
    fine = [0, 3, 5]
    check_norm(dq, h[fine], ref[fine], 320, fmt, s[fine], y[fine], sc[fine] if fmt else None)
    assert torch.isnan(y[1].float()).all()
    assert torch.isnan(y[2, 319].float()) and torch.isnan(y[4, 100].float())   # inf / inf
    assert torch.isnan(s[1, 3]) and s[2, 319] == float("inf") and s[4, 100] == float("-inf")
    if fmt:
        assert torch.isnan(sc[1]).all()
    if fmt == 1:
        assert torch.isnan(sc[2]).all() and torch.isnan(sc[4]).all()


@pytest.mark.parametrize("C", [96, 1000, 5120])
def test_norm_in_place(dq, C):
    """The residual stream updated where it lies, and BF16 rows normalised where they lie."""
    x, r, g = norm_input(9, C, True, True, seed=2)
    h, ref = norm_reference(x, r, g, 1e-6)
    xd, rd, gd = x.cuda(), r.cuda(), g.cuda()
    yd = torch.empty_like(xd)
    dq.dq_rmsnorm_forward(xd, 9, C, yd, residual=rd, sum_out=rd, gamma=gd)
    torch.cuda.synchronize()
    check_norm(dq, h, ref, C, 0, rd.cpu(), yd.cpu(), None)
    dq.dq_rmsnorm_forward(xd, 9, C, xd, residual=r.cuda(), gamma=gd)
    torch.cuda.synchronize()
    assert torch.equal(xd, yd)
    xd = x.cuda()
    dq.dq_rmsnorm_forward(xd, 9, C, yd, residual=r.cuda(), sum_out=xd, gamma=gd)
    torch.cuda.synchronize()
    assert torch.equal(xd, rd)


def test_norm_repeats_to_the_bit_and_replays(dq):
    x, r, g = (t.cuda() for t in norm_input(40, 5120, True, True))
    q = torch.zeros(40, 5120, dtype=torch.float8_e4m3fn, device="cuda")
    sc, sm = torch.zeros(40, 80, device="cuda"), torch.zeros_like(x)
    st = torch.cuda.Stream()
    call = lambda: dq.dq_rmsnorm_forward(x, 40, 5120, q, residual=r, sum_out=sm, gamma=g,  # noqa: E731
                                         y_format=dq.DQ_ROWS_E4M3_GROUP64, y_scales=sc, stream=st)
    st.wait_stream(torch.cuda.current_stream())
    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in (q.view(torch.uint8), sc, sm)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for t in (q, sc, sm):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (q.view(torch.uint8), sc, sm)):
        assert torch.equal(a, b)
    del graph


# ------------------------------------------------------------------ product of few rows

def run_rows(dq, dev, w, x, scales, fmt, gelu=False, x_pad=0, y_pad=0, ws=None, stream=None, status=0):
    rows = x.shape[0]
    xb = torch.zeros(rows, w.Ci + x_pad, dtype=x.dtype, device="cuda")
    xb[:, :w.Ci] = x.cuda()
    if x_pad:
        xb[:, w.Ci:] = float("nan")
    yb = torch.full((rows + 2, w.Co + y_pad), SENTINEL, dtype=torch.bfloat16, device="cuda")
    need = dq.dq_rows_workspace_bytes(rows, w.Ci, w.Co, w.rank)
    if ws is None:   # not cleared: nothing of the workspace's contents may matter
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    sc = scales.cuda() if scales is not None else None
    torch.cuda.synchronize()
    dq.dq_rows_forward(xb, rows, w.Ci, w.Co, w.rank, *dev, yb, ws, ws.numel(), x_stride=w.Ci + x_pad, x_format=fmt,
                       x_scales=sc, epilogue=dq.DQ_EPILOGUE_GELU if gelu else 0, y_stride=w.Co + y_pad, stream=stream)
    torch.cuda.synchronize()
    assert dq.dq_read_device_status(ws, stream) == status
    y = yb.cpu()
    assert (y[rows:] == SENTINEL).all() and (y[:, w.Co:] == SENTINEL).all()
    return y[:rows, :w.Co]


ROWS_LAYERS = [(256, 256, 16), (512, 768, 32), (1280, 256, 48), (256, 1024, 128), (2816, 512, 64)]


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("rows", [1, 2, 8, 15, 16, 17, 33, 64, 65, 77, 130])
@pytest.mark.parametrize("Ci,Co,rank", ROWS_LAYERS)
def test_rows(dq, Ci, Co, rank, rows, fmt):
    w, dev = weight(dq, Ci, Co, rank, seed=Ci, bias=Ci != 512)
    v, x, sc = rows_input(rows, Ci, fmt, seed=rows)
    gelu = (rows + fmt) % 2 == 1
    y = run_rows(dq, dev, w, x, sc, fmt, gelu=gelu, x_pad=16 * (rows % 3), y_pad=rows % 5)
    ref, tol = rows_reference(w, v, gelu)
    assert_within(y, ref, tol, "Y")


@pytest.mark.parametrize("rows", [255, 256, 257, 300, 513, 1000])
def test_more_rows(dq, rows):
    w, dev = weight(dq, 512, 768, 32, seed=512)
    for fmt in (0, 2):
        v, x, sc = rows_input(rows, 512, fmt, seed=rows)
        ref, tol = rows_reference(w, v, False)
        assert_within(run_rows(dq, dev, w, x, sc, fmt), ref, tol, "Y")


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_rows_c2_weight(dq, fmt):
    w, dev = weight(dq, 512, 512, 32, seed=4, c2=True, bias=True)
    v, x, sc = rows_input(5, 512, fmt)
    ref, tol = rows_reference(w, v, False)
    assert_within(run_rows(dq, dev, w, x, sc, fmt), ref, tol, "Y")


@pytest.mark.parametrize("rows", [1, 9, 70])
def test_rows_wide_layer(dq, rows):
    """A layer with many tiles along both sides."""
    w, dev = weight(dq, 5120, 2816, 32, seed=8, bias=True)
    for fmt in (0, 1, 2):
        v, x, sc = rows_input(rows, 5120, fmt, seed=rows)
        ref, tol = rows_reference(w, v, fmt == 1)
        assert_within(run_rows(dq, dev, w, x, sc, fmt, gelu=fmt == 1), ref, tol, "Y")


def test_rows_of_any_magnitude(dq):
    """BF16 rows from 2^-110 to 2^100, zeros, and 30 binades within a row: the bound is relative to each row."""
    w, dev = weight(dq, 512, 768, 32, seed=512)
    v, x, _ = rows_input(8, 512, 0, seed=1)
    v = v.clone()
    for m, e in enumerate((-110, 100, -60, 40)):
        v[m] = torch.ldexp(v[m], torch.tensor(e))
    v[4] = 0
    v[5] = torch.ldexp(v[5], torch.arange(512) % 31 - 15)
    x = bf16(v)
    v = x.double()
    ref, tol = rows_reference(w, v, False)
    # a product below BF16's normal range rounds to steps of 2^-133
    assert_within(run_rows(dq, dev, w, x, None, 0), ref, tol, "Y")


def test_rows_not_finite_stay_alone(dq):
    w, dev = weight(dq, 512, 768, 32, seed=512)
    for rows in (5, 70):
        v, x, _ = rows_input(rows, 512, 0)
        x[1, 7], x[3, 500] = float("nan"), float("inf")
        y = run_rows(dq, dev, w, x, None, 0)
        assert torch.isnan(y[1].float()).all() and torch.isnan(y[3].float()).all()
        fine = [m for m in range(rows) if m not in (1, 3)]
        ref, tol = rows_reference(w, v, False)
        assert_within(y[fine], ref[fine], tol[fine], "Y")
    v, x, sc = rows_input(3, 512, 1)
    x.view(torch.uint8)[1, 9] = 0x7F
    sc[2] = float("nan")
    y = run_rows(dq, dev, w, x, sc, 1)
    assert torch.isnan(y[1:].float()).all()
    ref, tol = rows_reference(w, v, False)
    assert_within(y[:1], ref[:1], tol[:1], "Y")


def test_rows_with_zero_scales(dq):
    """Rows, and groups of rows, that were quantised from zeros."""
    w, dev = weight(dq, 512, 512, 32, seed=4, c2=True, bias=True)
    for fmt in (1, 2):
        x = torch.randn(4, 512, generator=torch.Generator().manual_seed(3))
        x[1], x[2, 64:192] = 0, 0
        v, q, sc = quantise_rows(x, fmt)
        ref, tol = rows_reference(w, v, False)
        y = run_rows(dq, dev, w, q, sc, fmt)
        assert_within(y, ref, tol, "Y")
        assert torch.equal(y[1], w.bias)


def test_rows_share_a_larger_workspace_in_turn(dq):
    """One workspace, sized for the most rows, serves calls of other layers and row counts one after another."""
    ws = torch.zeros(dq.dq_rows_workspace_bytes(130, 1280, 768, 64), dtype=torch.uint8, device="cuda")
    for Ci, Co, rank, rows in ((512, 768, 32, 130), (1280, 256, 48, 3), (512, 768, 32, 17), (256, 256, 16, 130)):
        w, dev = weight(dq, Ci, Co, rank, seed=Ci, bias=Ci != 512)
        v, x, sc = rows_input(rows, Ci, 0, seed=rows)
        ref, tol = rows_reference(w, v, False)
        assert_within(run_rows(dq, dev, w, x, sc, 0, ws=ws), ref, tol, "Y")


def test_rows_report_a_bad_packed_weight(dq):
    w, dev = weight(dq, 512, 768, 32, seed=512)
    v, x, _ = rows_input(3, 512, 0)
    bad = dev[0].clone()
    bad[0] ^= 0xFF
    y = run_rows(dq, (bad, *dev[1:]), w, x, None, 0, status=dq.DQ_ERR_BAD_PACKED_WEIGHT)
    assert (y == SENTINEL).all()
    # the packed weight of a layer with other sizes
    other, _ = weight(dq, 256, 1024, 128, seed=256, bias=True)
    big = torch.zeros(w.packed.size, dtype=torch.uint8)
    big[:256] = torch.from_numpy(other.packed[:256])
    y = run_rows(dq, (big.cuda(), *dev[1:]), w, x, None, 0, status=dq.DQ_ERR_BAD_PACKED_WEIGHT)
    assert (y == SENTINEL).all()
    ws = torch.zeros(dq.dq_rows_workspace_bytes(3, 512, 768, 32), dtype=torch.uint8, device="cuda")
    run_rows(dq, (bad, *dev[1:]), w, x, None, 0, ws=ws, status=dq.DQ_ERR_BAD_PACKED_WEIGHT)
    ref, tol = rows_reference(w, v, False)
    assert_within(run_rows(dq, dev, w, x, None, 0, ws=ws), ref, tol, "Y")   # the next call clears it


@pytest.mark.parametrize("rows", [1, 24, 80])
def test_rows_repeat_to_the_bit_and_replay(dq, rows):
    """Calls one after another without a wait, and a captured call with new inputs copied into its buffers."""
    w, dev = weight(dq, 2816, 512, 64, seed=2816, bias=True)
    _, x0, _ = rows_input(rows, 2816, 0, seed=1)
    _, x1, _ = rows_input(rows, 2816, 0, seed=2)
    want = [run_rows(dq, dev, w, x, None, 0, gelu=True) for x in (x0, x1)]
    st = torch.cuda.Stream()
    need = dq.dq_rows_workspace_bytes(rows, 2816, 512, 64)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    xs = [x0.cuda(), x1.cuda()]
    ys = [torch.zeros(rows, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    xg = xs[0].clone()
    torch.cuda.synchronize()

    def call(x, y):
        dq.dq_rows_forward(x, rows, 2816, 512, 64, *dev, y, ws, need, epilogue=dq.DQ_EPILOGUE_GELU, stream=st)

    for _ in range(20):
        call(xs[0], ys[0])
        call(xs[1], ys[1])
    torch.cuda.synchronize()
    assert all(torch.equal(y.cpu(), r) for y, r in zip(ys, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call(xg, ys[0])
    for i in (1, 0, 1):
        xg.copy_(xs[i])
        ys[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0].cpu(), want[i])
    assert dq.dq_read_device_status(ws, st) == 0
    del graph


def test_rows_on_two_streams(dq):
    """Calls that overlap on two streams, each with a workspace of its own."""
    w, dev = weight(dq, 2816, 512, 64, seed=2816, bias=True)
    xs, ys, wss, want = [], [], [], []
    for i, rows in enumerate((3, 40)):
        _, x, _ = rows_input(rows, 2816, 0, seed=i)
        want.append(run_rows(dq, dev, w, x, None, 0))
        xs.append(x.cuda())
        ys.append(torch.zeros(rows, 512, dtype=torch.bfloat16, device="cuda"))
        wss.append(torch.zeros(dq.dq_rows_workspace_bytes(rows, 2816, 512, 64), dtype=torch.uint8, device="cuda"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            dq.dq_rows_forward(xs[i], xs[i].shape[0], 2816, 512, 64, *dev, ys[i], wss[i], wss[i].numel(),
                               stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(y.cpu(), r) for y, r in zip(ys, want))


# ------------------------------------------------------------------ cuts of the product, order of launches

@pytest.mark.parametrize("rows", range(1, 10))
@pytest.mark.parametrize("Ci,Co,rank", [(256, 1280, 112), (1536, 2560, 32), (7168, 256, 16), (5120, 768, 80)])
def test_few_rows_of_every_count(dq, Ci, Co, rank, rows):
    """One row to one more than a single launch takes, in layers that are cut into clusters in different ways."""
    w, dev = weight(dq, Ci, Co, rank, seed=Ci, bias=True)
    for fmt in (0, 1, 2):
        v, x, sc = rows_input(rows, Ci, fmt, seed=10 * rows + fmt)
        ref, tol = rows_reference(w, v, fmt == 2)
        assert_within(run_rows(dq, dev, w, x, sc, fmt, gelu=fmt == 2, y_pad=rows % 2), ref, tol, "Y")


@pytest.mark.parametrize("Ci,Co,rank,rows", [(256, 20480, 16, 9), (256, 20480, 112, 17), (512, 20480, 32, 64), (256, 5120, 128, 130),
                                             (768, 5120, 48, 155), (1280, 5120, 64, 310), (512, 2560, 32, 1001), (256, 256, 16, 4740)])
def test_rows_with_more_work_than_fits_at_once(dq, Ci, Co, rank, rows):
    """Layers of many tiles and many rows, odd counts of them in a pass."""
    w, dev = weight(dq, Ci, Co, rank, seed=Ci + Co, bias=True)
    for fmt in (0, 1, 2):
        v, x, sc = rows_input(rows, Ci, fmt, seed=rows + fmt)
        ref, tol = rows_reference(w, v, fmt == 1)
        assert_within(run_rows(dq, dev, w, x, sc, fmt, gelu=fmt == 1, x_pad=16, y_pad=3), ref, tol, "Y")


@pytest.mark.parametrize("fmt", [0, 2])
def test_the_most_rows(dq, fmt):
    """As many rows as a call takes, a few of them not finite, in the smallest layer."""
    rows = 65535
    w, dev = weight(dq, 256, 256, 16, seed=256, bias=True)
    v, x, sc = rows_input(rows, 256, fmt, seed=1)
    bad = [0, 31, 4096, rows - 1]
    if fmt == 0:
        x[bad, 77] = float("nan")
    else:
        sc[bad, 1] = float("inf")
    y = run_rows(dq, dev, w, x, sc, fmt, x_pad=16)
    ref, tol = rows_reference(w, v, False)
    assert torch.isnan(y[bad].float()).all()
    fine = torch.ones(rows, dtype=torch.bool)
    fine[bad] = False
    assert_within(y[fine], ref[fine], tol[fine], "Y")


@pytest.mark.parametrize("rows", [4, 40])
def test_rows_with_scales_that_are_not_finite(dq, rows):
    w, dev = weight(dq, 512, 768, 32, seed=512)
    v, x, sc = rows_input(rows, 512, 1)
    sc[0], sc[2] = float("inf"), float("-inf")
    y = run_rows(dq, dev, w, x, sc, 1)
    ref, tol = rows_reference(w, v, False)
    fine = [m for m in range(rows) if m not in (0, 2)]
    assert torch.isnan(y[0].float()).all() and torch.isnan(y[2].float()).all()
    assert_within(y[fine], ref[fine], tol[fine], "Y")
    v, x, sc = rows_input(rows, 512, 2)
    sc[1, 3] = float("inf")
    y = run_rows(dq, dev, w, x, sc, 2)
    ref, tol = rows_reference(w, v, False)
    fine = [m for m in range(rows) if m != 1]
    assert torch.isnan(y[1].float()).all()
    assert_within(y[fine], ref[fine], tol[fine], "Y")


@pytest.mark.parametrize("rows", [1, 8, 30])
def test_a_chain_without_waits_is_the_chain_with_waits(dq, rows):
    """Blocks one after another on one stream, each on the output of the one before, all through the same buffers:
    every launch has to wait for what it reads and for the readers of what it writes."""
    C, F = 512, 1024
    _, updev = weight(dq, C, F, 32, seed=21, bias=True)
    _, downdev = weight(dq, F, C, 48, seed=22, bias=True)
    x, r, g = norm_input(rows, C, True, True, seed=rows)
    gd, st = g.cuda(), torch.cuda.Stream()
    ws = torch.zeros(max(dq.dq_rows_workspace_bytes(rows, C, F, 32), dq.dq_rows_workspace_bytes(rows, F, C, 48)),
                     dtype=torch.uint8, device="cuda")
    q, sd = torch.zeros(rows, C, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(rows, C // 64, device="cuda")
    hid = torch.zeros(rows, F, dtype=torch.bfloat16, device="cuda")
    ends = []
    for wait in (True, False, False):
        y, res = x.cuda(), r.cuda()
        torch.cuda.synchronize()
        for _ in range(12):
            for step in range(3):
                if step == 0:
                    dq.dq_rmsnorm_forward(y, rows, C, q, residual=res, sum_out=res, gamma=gd,
                                          y_format=dq.DQ_ROWS_E4M3_GROUP64, y_scales=sd, stream=st)
                elif step == 1:
                    dq.dq_rows_forward(q, rows, C, F, 32, *updev, hid, ws, ws.numel(), x_format=dq.DQ_ROWS_E4M3_GROUP64,
                                       x_scales=sd, epilogue=dq.DQ_EPILOGUE_GELU, stream=st)
                else:
                    dq.dq_rows_forward(hid, rows, F, C, 48, *downdev, y, ws, ws.numel(), stream=st)
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert dq.dq_read_device_status(ws, st) == 0
        ends.append((y.cpu(), res.cpu()))
    assert torch.isfinite(ends[0][0].float()).all()
    for y, res in ends[1:]:
        assert torch.equal(y, ends[0][0]) and torch.equal(res, ends[0][1])


def test_two_captured_calls_with_workspaces_of_their_own_overlap(dq):
    w, dev = weight(dq, 2816, 512, 64, seed=2816, bias=True)
    graphs, ys, want = [], [], []
    for i, rows in enumerate((5, 33)):
        _, x, _ = rows_input(rows, 2816, 0, seed=40 + i)
        want.append(run_rows(dq, dev, w, x, None, 0))
        xd, st, graph = x.cuda(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        ys.append(torch.zeros(rows, 512, dtype=torch.bfloat16, device="cuda"))
        ws = torch.zeros(dq.dq_rows_workspace_bytes(rows, 2816, 512, 64), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            for _ in range(3):
                dq.dq_rows_forward(xd, rows, 2816, 512, 64, *dev, ys[i], ws, ws.numel(), stream=st)
        graphs.append((graph, st, xd, ws))
    for _ in range(5):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for graph, st, _, _ in graphs:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y.cpu(), r) for y, r in zip(ys, want))
    graphs.clear()


FIRST_CALL = """
import sys
import torch
import video_diffusion_w4a4_b200 as dq
from rows_case import Weight, rows_input
rows, fmt = int(sys.argv[1]), 1
w = Weight(dq, 512, 768, 32, seed=3, bias=True)
dev = w.device()
_, x, sc = rows_input(rows, 512, fmt, seed=4)
xd, sd = x.cuda(), sc.cuda()
h = torch.ones(rows, 768, dtype=torch.bfloat16, device="cuda")
y, n = torch.zeros_like(h), torch.zeros_like(h)
ws = torch.zeros(dq.dq_rows_workspace_bytes(rows, 512, 768, 32), dtype=torch.uint8, device="cuda")
st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()


def calls():
    dq.dq_rows_forward(xd, rows, 512, 768, 32, *dev, y, ws, ws.numel(), x_format=fmt, x_scales=sd, stream=st)
    dq.dq_rmsnorm_forward(y, rows, 768, n, residual=h, stream=st)


with torch.cuda.graph(graph, stream=st):
    calls()
graph.replay()
torch.cuda.synchronize()
first = y.clone(), n.clone()
y.zero_(), n.zero_()
calls()
torch.cuda.synchronize()
assert torch.equal(first[0], y) and torch.equal(first[1], n) and bool((y != 0).any())
del graph
print("captured first")
"""


@pytest.mark.parametrize("rows", [2, 20])
def test_the_first_call_of_a_process_may_be_captured(rows):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([root, os.path.join(root, "tests"), os.environ.get("PYTHONPATH", "")]))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL, str(rows)], env=env, cwd=root, capture_output=True, text=True,
                         timeout=240)
    assert out.returncode == 0 and "captured first" in out.stdout, out.stdout + out.stderr


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("rows", [1, 21])
def test_block_of_few_rows(dq, rows, fmt):
    """A feed-forward block of few rows: the residual's addition and the norm, the up-projection with GELU on
    its (8-bit) output, the down-projection.  Each step against its definition on the step before's output."""
    C, F = 512, 1024
    up, updev = weight(dq, C, F, 32, seed=21, bias=True)
    down, downdev = weight(dq, F, C, 48, seed=22, bias=True)
    x, r, g = norm_input(rows, C, True, True, seed=rows)
    st = torch.cuda.Stream()
    xd, rd, gd = x.cuda(), r.cuda(), g.cuda()
    qd = torch.zeros(rows, C, dtype=torch.bfloat16 if fmt == 0 else torch.float8_e4m3fn, device="cuda")
    sd = torch.zeros(rows, 1 if fmt == 1 else C // 64, device="cuda") if fmt else None
    hid = torch.zeros(rows, F, dtype=torch.bfloat16, device="cuda")
    yd = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(max(dq.dq_rows_workspace_bytes(rows, C, F, 32), dq.dq_rows_workspace_bytes(rows, F, C, 48)),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    dq.dq_rmsnorm_forward(xd, rows, C, qd, residual=rd, sum_out=rd, gamma=gd, y_format=fmt, y_scales=sd, stream=st)
    dq.dq_rows_forward(qd, rows, C, F, 32, *updev, hid, ws, ws.numel(), x_format=fmt, x_scales=sd,
                       epilogue=dq.DQ_EPILOGUE_GELU, stream=st)
    dq.dq_rows_forward(hid, rows, F, C, 48, *downdev, yd, ws, ws.numel(), stream=st)
    torch.cuda.synchronize()
    h, y = norm_reference(x, r, g, 1e-6)
    check_norm(dq, h, y, C, fmt, rd.cpu(), qd.cpu(), sd.cpu() if fmt else None)
    v = qd.cpu().double()
    if fmt:
        v = v * sd.cpu().double().repeat_interleave(C // sd.shape[1], 1)
    ref, tol = rows_reference(up, v, True)
    assert_within(hid, ref, tol, "hidden")
    ref, tol = rows_reference(down, hid.cpu().double(), False)
    assert_within(yd, ref, tol, "Y")


def test_norm_before_a_cube_layer(dq):
    """BF16 rows of the norm as the input of the 4-bit cube layer, in order on one stream."""
    import oracle
    import synth
    from dq_case import Case, assert_y_close, compare_quantised
    wl = synth.Workload("norm_cube", 3, 4, 8, 512, 256, 32, (1, 2, 2), (3, 1, 2), (0.01, 50.0), (0.01, 20.0))
    case = Case(wl)
    x = torch.from_numpy(case.X.view(np.int16).copy()).view(torch.bfloat16)
    _, r, g = norm_input(wl.N, wl.Ci, True, True, seed=6)
    xd, y = x.cuda(), torch.empty(wl.N, wl.Ci, dtype=torch.bfloat16, device="cuda")
    dq.dq_rmsnorm_forward(xd, wl.N, wl.Ci, y, residual=r.cuda(), gamma=g.cuda())
    torch.cuda.synchronize()
    h, ref = norm_reference(x, r, g, 1e-6)
    check_norm(dq, h, ref, wl.Ci, 0, None, y.cpu(), None)
    case.X = y.cpu().view(torch.int16).numpy().view(np.uint16)
    got = case.run_gpu(dq, torch)
    act, wq = case.run_oracle()
    compare_quantised(got, act, wq)
    assert_y_close(got["Y"], case.oracle_rows(act, wq, np.arange(wl.N)))
