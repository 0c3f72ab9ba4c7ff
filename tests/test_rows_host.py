"""Argument checks of the few-row operators (no GPU): every refusal comes before any device call."""
import numpy as np
import pytest

import video_diffusion_w4a4_b200 as dq

P = 1 << 20   # a 256-byte-aligned stand-in address; nothing is dereferenced on these paths


def norm(x=P, xs=0, r=P, rs=0, g=P, rows=4, C=512, eps=1e-6, so=P, ss=0, fmt=0, y=P, ys=0, sc=None):
    return dq._lib.dq_rmsnorm_forward(x, xs, r, rs, g, rows, C, eps, so, ss, fmt, y, ys, sc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "INVALID_ARG"), (dict(C=0), "INVALID_ARG"), (dict(eps=-1e-6), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"), (dict(fmt=3), "INVALID_ARG"),
    (dict(C=32769), "UNSUPPORTED_SHAPE"), (dict(rows=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(xs=511), "INVALID_ARG"), (dict(rs=511), "INVALID_ARG"), (dict(ss=511), "INVALID_ARG"),
    (dict(ys=-512), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"),
    (dict(fmt=1), "INVALID_ARG"), (dict(fmt=0, sc=P), "INVALID_ARG"), (dict(x=P + 1), "ALIGNMENT"),
    (dict(r=P + 1), "ALIGNMENT"), (dict(g=P + 1), "ALIGNMENT"), (dict(so=P + 1), "ALIGNMENT"),
    (dict(y=P + 1), "ALIGNMENT"), (dict(fmt=2, sc=P + 2), "ALIGNMENT")])
def test_norm_refusals(kw, code):
    assert norm(**kw) == getattr(dq, "DQ_ERR_" + code)


def test_norm_of_no_rows_does_nothing():
    assert norm(rows=0) == dq.DQ_OK
    assert norm(rows=0, x=None, y=None, r=None, g=None, so=None) == dq.DQ_OK


def rows(x=P, fmt=0, xs=0, sc=None, m=4, Ci=512, Co=256, r=32, w=P, l1=P, l2=P, epi=0, y=P, ys=0, ws=P, wsb=1 << 40):
    return dq._lib.dq_rows_forward(x, fmt, xs, sc, m, Ci, Co, r, w, l1, l2, epi, y, ys, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), "INVALID_ARG"), (dict(m=65536), "UNSUPPORTED_SHAPE"), (dict(Ci=384), "UNSUPPORTED_SHAPE"),
    (dict(Co=100), "UNSUPPORTED_SHAPE"), (dict(r=8), "UNSUPPORTED_SHAPE"), (dict(r=144), "UNSUPPORTED_SHAPE"),
    (dict(fmt=3), "INVALID_ARG"), (dict(fmt=-1), "INVALID_ARG"), (dict(epi=2), "INVALID_ARG"),
    (dict(fmt=1), "INVALID_ARG"), (dict(fmt=0, sc=P), "INVALID_ARG"), (dict(xs=504), "INVALID_ARG"),
    (dict(ys=255), "INVALID_ARG"), (dict(xs=516), "ALIGNMENT"), (dict(fmt=1, sc=P, xs=520), "ALIGNMENT"),
    (dict(x=P + 8), "ALIGNMENT"), (dict(fmt=2, sc=P + 2), "ALIGNMENT"), (dict(y=P + 1), "ALIGNMENT"),
    (dict(w=P + 128), "ALIGNMENT"), (dict(l1=P + 128), "ALIGNMENT"), (dict(l2=P + 128), "ALIGNMENT"),
    (dict(ws=P + 128), "ALIGNMENT"), (dict(wsb=16), "WORKSPACE_TOO_SMALL"), (dict(x=None), "INVALID_ARG"),
    (dict(w=None), "INVALID_ARG"), (dict(l1=None), "INVALID_ARG"), (dict(l2=None), "INVALID_ARG"),
    (dict(y=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG")])
def test_rows_refusals(kw, code):
    assert rows(**kw) == getattr(dq, "DQ_ERR_" + code)


def test_rows_of_none_does_nothing():
    assert rows(m=0) == dq.DQ_OK
    assert rows(m=0, x=None, y=None, ws=None, wsb=0) == dq.DQ_OK


def test_rows_workspace_grows_with_rows_and_is_checked_to_the_byte():
    sizes = [dq.dq_rows_workspace_bytes(m, 5120, 5120, 32) for m in (0, 1, 2, 16, 17, 64, 65, 256, 257, 512, 65535)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
    need = dq.dq_rows_workspace_bytes(4, 512, 256, 32)
    assert rows(wsb=need - 1) == dq.DQ_ERR_WORKSPACE_TOO_SMALL
    for bad in ((-1, 512, 256, 32), (4, 500, 256, 32), (4, 512, 256, 20)):
        with pytest.raises(dq.DQError):
            dq.dq_rows_workspace_bytes(*bad)


def test_python_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(1, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dq.dq_rmsnorm_forward(x, 1, 256, x)
    with pytest.raises(ValueError):
        dq.dq_rows_forward(x, 1, 256, 256, 16, x, x, x, x, x, 1 << 20)


def test_reference_decodes_the_packed_weight():
    """The tests' own 64-bit weight against the packer's BF16 copy of q s_b (another section of the blob)."""
    from rows_case import Weight
    w = Weight(dq, 512, 256, 16, seed=3)
    lay = dq.dq_packed_weight_layout(256, 512, 16)
    d = w.packed[lay.off_dqw:lay.off_dqw + 256 * 512 * 2].view(np.uint16).astype(np.uint32) << 16
    s_w = float(w.packed[24:28].view(np.float32)[0])
    assert np.array_equal(d.view(np.float32).astype(np.float64).reshape(256, 512) * s_w, w.values)


def test_rows_wait_selftest_refusals():
    call = lambda us=50000, m=4: dq._lib.dq_selftest_rows_wait(us, P, m, 512, 256, 32, P, P, P, P, P, 16, None)  # noqa: E731
    assert call(us=999) == dq.DQ_ERR_INVALID_ARG and call(m=0) == dq.DQ_ERR_INVALID_ARG
    assert call() == dq.DQ_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("eps", [0.0, 1e-6, 3.3e38])
def test_norm_takes_every_finite_eps(eps):
    assert norm(rows=0, eps=eps) == dq.DQ_OK
