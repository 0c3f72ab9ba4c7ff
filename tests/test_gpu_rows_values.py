"""dq_rows_forward on rows whose values span many binades: what the large values leave to an output whose weights are
zero there is held to the bound of include/deltaquant.h (a value is off by 2^-23 of its row's largest at most, an
eighth of a row's values by more than 2^-9 of themselves, else the row is summed in fp32)."""
import numpy as np
import pytest
import torch

from rows_case import U, Weight, assert_within, bf16, quantise_rows, w_t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    import video_diffusion_w4a4_b200 as m
    return m


_weights = {}


def blind_weight(dq, Ci, Co, rank, channels):
    """A packed layer that does not read the input channels given: their codes are 0 and so are their rows of L1."""
    key = (Ci, Co, rank, tuple(channels))
    if key not in _weights:
        w = Weight(dq, Ci, Co, rank, seed=Ci + Co, bias=True)
        lay = dq.dq_packed_weight_layout(Co, Ci, rank)
        codes = w.packed[lay.off_codes:lay.off_codes + Co * Ci // 2].reshape(Co, Ci // 2)
        for c in channels:
            codes[:, c // 2] &= 0xF0 if c % 2 == 0 else 0x0F
            w.values[:, c] = 0
            w.l1[c] = 0
            w._host[1].reshape(rank, Ci)[:, c] = 0
        _weights[key] = (w, w.device())
    return _weights[key]


def wide_rows(rows, Ci, fmt, binades, channels, seed):
    """Rows of normal values with 1.5 2^binades in the channels given, as (values in 64 bits, tensor, scales)."""
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((rows, Ci)))
    x[:, channels] = 1.5 * 2.0 ** binades
    if fmt == 0:
        xb = bf16(x)
        return xb.double(), xb, None
    return quantise_rows(x, fmt)


def reference(w, v, fmt):
    """(Y, tolerance): the terms of rows_case.rows_reference, with the digits' rounding only as far as the header has it."""
    wv, l1, l2, b = torch.from_numpy(w.values), w.l1.double(), w.l2.double(), w.bias.double()
    y = v @ w_t(wv) + (v @ l1) @ l2 + b
    A, B = v.abs() @ w_t(wv.abs()) + b.abs(), (v.abs() @ l1.abs()) @ l2.abs()
    M = v.abs().amax(1, keepdim=True)
    T = 2.0 ** (torch.floor(torch.log2(M)) - 15)
    lossy = (v != 0) & (v.abs() < T)
    part = lossy.sum(1) / (v != 0).sum(1)
    assert ((part < 0.09) | (part > 0.2)).all()   # clearly on one side, in each part of the channels too
    off = 2.0 ** -23 * M * (lossy if fmt == 0 else (v != 0) & (fmt == 2)) * (part <= 0.125)[:, None]
    tol = off @ w_t(wv.abs()) + 2 * U * (w.Ci / 16 + 32) * A + (2 * U * (w.Ci / 16 + 2 * w.rank + 32) + 2.0 ** -16) * B
    return y, tol + 2.0 ** -8 * y.abs() + 2.0 ** -133


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("binades", [0, 9, 14, 17, 20, 24, 60])
@pytest.mark.parametrize("Ci,Co,rank,rows", [(512, 768, 32, 1), (512, 768, 32, 3), (512, 768, 32, 8), (512, 768, 32, 70),
                                             (5120, 768, 80, 4), (5120, 768, 80, 21), (768, 5120, 48, 155),
                                             (8448, 256, 16, 2), (8448, 256, 16, 11)])
def test_small_values_beside_large_ones_that_no_output_reads(dq, Ci, Co, rank, rows, binades, fmt):
    channels = [Ci // 2 + 5]
    w, dev = blind_weight(dq, Ci, Co, rank, channels)
    v, x, sc = wide_rows(rows, Ci, fmt, binades, channels, seed=rows + binades)
    if fmt == 1 and binades > 9:   # one scale a row leaves E4M3 codes of nothing else
        v, x, sc = wide_rows(rows, Ci, fmt, 9, channels, seed=rows + binades)
    y = torch.full((rows + 1, Co), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((dq.dq_rows_workspace_bytes(rows, Ci, Co, rank),), 0xFF, dtype=torch.uint8, device="cuda")
    dq.dq_rows_forward(x.cuda(), rows, Ci, Co, rank, *dev, y, ws, ws.numel(), x_format=fmt,
                       x_scales=sc.cuda() if fmt else None)
    torch.cuda.synchronize()
    assert dq.dq_read_device_status(ws) == 0 and (y[rows:] == -7).all()
    ref, tol = reference(w, v, fmt)
    assert_within(y[:rows], ref, tol, "Y")


@pytest.mark.parametrize("fmt", [0, 2])
@pytest.mark.parametrize("Ci,Co,rank,rows", [(512, 768, 32, 8), (1280, 768, 32, 41), (768, 5120, 48, 155)])
def test_rows_of_both_kinds_in_one_call(dq, Ci, Co, rank, rows, fmt):
    """Every third row spans more than the others, one is not finite: each gives what it gives in a call of its own kind."""
    channels = [3, Ci - 1]
    w, dev = blind_weight(dq, Ci, Co, rank, channels)
    x = torch.from_numpy(np.random.default_rng(rows).standard_normal((rows, Ci)))
    x[::3, channels] = 1.5 * 2.0 ** 19
    if fmt == 0:
        x = bf16(x)
        v, sc = x.double(), None
    else:
        v, x, sc = quantise_rows(x, fmt)
    bad = rows // 2
    if fmt == 0:
        x[bad, 9] = float("inf")
    else:
        sc[bad, 1] = float("nan")
    y = torch.empty(rows, Co, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((dq.dq_rows_workspace_bytes(rows, Ci, Co, rank),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):   # one call after another through the same workspace
        dq.dq_rows_forward(x.cuda(), rows, Ci, Co, rank, *dev, y, ws, ws.numel(), x_format=fmt,
                           x_scales=sc.cuda() if fmt else None)
    torch.cuda.synchronize()
    assert dq.dq_read_device_status(ws) == 0
    assert torch.isnan(y[bad].float()).all()
    fine = [m for m in range(rows) if m != bad]
    ref, tol = reference(w, v[fine], fmt)
    assert_within(y[fine], ref, tol, "Y")


def test_values_at_the_ends_of_the_range(dq):
    """Rows from BF16's largest values to its smallest at once, where neither unit nor sums may overflow."""
    channels = [100, 101]
    w, dev = blind_weight(dq, 512, 768, 32, channels)
    x = torch.from_numpy(np.random.default_rng(5).standard_normal((9, 512)))
    x[0] *= 2.0 ** 100
    x[0, 100], x[0, 101] = 3e38, -3e38
    x[1] *= 2.0 ** -100
    x[1, 100] = 1.0
    x[2] = torch.ldexp(x[2], torch.arange(512) % 120 - 60)
    x[2, 100] = 2.0 ** 90
    x[3] *= 2.0 ** -120
    x[3, 101] = 2.0 ** -90
    x = bf16(x)
    for rows in (4, 9):
        y = torch.empty(rows, 768, dtype=torch.bfloat16, device="cuda")
        ws = torch.full((dq.dq_rows_workspace_bytes(rows, 512, 768, 32),), 0xFF, dtype=torch.uint8, device="cuda")
        dq.dq_rows_forward(x[:rows].cuda(), rows, 512, 768, 32, *dev, y, ws, ws.numel())
        torch.cuda.synchronize()
        ref, tol = reference(w, x[:rows].double(), 0)
        assert_within(y, ref, tol, "Y")


@pytest.mark.parametrize("Ci,Co,rank,rows", [(512, 768, 32, 1), (512, 768, 32, 8), (512, 768, 32, 20), (768, 5120, 48, 155),
                                             (8448, 256, 16, 2)])
def test_of_a_weight_that_does_not_match_only_the_header_is_read(dq, Ci, Co, rank, rows):
    """A blob of 256 bytes, as a smaller layer's may end behind what this call's sizes point to; wide rows among the
    others.  A right weight at the same address is taken by the next call."""
    w, dev = blind_weight(dq, Ci, Co, rank, [Ci // 2 + 5])
    v, x, _ = wide_rows(rows, Ci, 0, 20, [Ci // 2 + 5], seed=rows)
    other, _ = blind_weight(dq, 256, 256, 16, [1])
    ws = torch.full((dq.dq_rows_workspace_bytes(rows, Ci, Co, rank),), 0xFF, dtype=torch.uint8, device="cuda")
    for head in (torch.from_numpy(other.packed[:256].copy()).cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")):
        y = torch.full((rows, Co), -7.0, dtype=torch.bfloat16, device="cuda")
        dq.dq_rows_forward(x.cuda(), rows, Ci, Co, rank, head, *dev[1:], y, ws, ws.numel())
        torch.cuda.synchronize()
        assert dq.dq_read_device_status(ws) == dq.DQ_ERR_BAD_PACKED_WEIGHT
        assert (y == -7).all()
    blob = torch.zeros_like(dev[0])
    xd, y = x.cuda(), torch.full((rows, Co), -7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    dq.dq_rows_forward(xd, rows, Ci, Co, rank, blob, *dev[1:], y, ws, ws.numel())
    blob.copy_(dev[0])
    dq.dq_rows_forward(xd, rows, Ci, Co, rank, blob, *dev[1:], y, ws, ws.numel())
    torch.cuda.synchronize()
    assert dq.dq_read_device_status(ws) == 0
    ref, tol = reference(w, v, 0)
    assert_within(y, ref, tol, "Y")


@pytest.mark.parametrize("Ci,Co,rank,rows", [(512, 768, 32, 1), (5120, 768, 80, 4), (1280, 2560, 32, 8)])
def test_a_wait_that_runs_out_leaves_y_and_is_reported(dq, Ci, Co, rank, rows):
    """The exchange of the low-rank sums waits for an arrival that never comes: the wait ends by its budget, the status
    word says so whatever it was before, and Y stays as it was.  The next call is as ever."""
    w, dev = blind_weight(dq, Ci, Co, rank, [5])
    v, x, _ = wide_rows(rows, Ci, 0, 0, [5], seed=rows)
    xd, y = x.cuda(), torch.full((rows, Co), -7.0, dtype=torch.bfloat16, device="cuda")
    need = dq.dq_rows_workspace_bytes(rows, Ci, Co, rank)
    for before in (0x00, 0xFF):
        ws = torch.full((need,), before, dtype=torch.uint8, device="cuda")
        dq.dq_selftest_rows_wait(50000, xd, rows, Ci, Co, rank, *dev, y, ws, need)
        torch.cuda.synchronize()
        assert dq.dq_read_device_status(ws) == dq.DQ_ERR_DEVICE_TIMEOUT
        assert (y == -7).all()
    dq.dq_rows_forward(xd, rows, Ci, Co, rank, *dev, y, ws, need)
    torch.cuda.synchronize()
    assert dq.dq_read_device_status(ws) == 0
    ref, tol = reference(w, v, 0)
    assert_within(y, ref, tol, "Y")
