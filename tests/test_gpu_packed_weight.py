"""The cube layers with a packed weight that is not this call's: reported, Y left as it was, nothing but the header read."""
import numpy as np
import pytest

import synth
from dq_case import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    import video_diffusion_w4a4_b200 as dq
    return dq, torch


def run(dq, torch, case, packed, **opts):
    wl, (t, h, w) = case.wl, case.cube
    _, L1m, L2s, _ = dq.dq_pack_weight_factors(case.Wb, case.L1, case.L2)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    X, P, L1, L2 = dev(case.X.view(np.int16)), dev(packed), dev(L1m.view(np.int16)), dev(L2s.view(np.int16))
    Y = torch.full((wl.N, wl.Co), -7.0, dtype=torch.bfloat16, device="cuda")
    lay = dq.dq_workspace_layout_opts(wl.T, wl.H, wl.W, t, h, w, wl.Ci, wl.Co, wl.rank, **opts)
    ws = torch.zeros(lay.total_bytes, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream()
    dq.dq_linear_forward_opts(X, wl.T, wl.H, wl.W, t, h, w, wl.Ci, wl.Co, wl.rank, P, L1, L2, Y, ws, lay.total_bytes, 7, None,
                              st, **opts)
    torch.cuda.synchronize()
    return dq.dq_read_device_status(ws, st), Y.float()


def header(dq, Co, Ci, rank, fp8):
    z = lambda r, c: np.zeros((r, c), np.uint16)  # noqa: E731
    packed, _, _, _ = dq.dq_pack_weight_factors(z(Co, Ci), z(Ci, rank), z(rank, Co), pack_flags=dq.DQ_PACK_C2 if fp8 else 0)
    return packed[:256].copy()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("sizes", [(512, 0), (0, 512)])
def test_a_weight_of_other_sizes(env, sizes, fp8):
    """The header says another Co, or another Ci."""
    dq, torch = env
    case = Case(synth.WORKLOADS["tiny"])
    wl = case.wl
    Co, Ci = sizes[0] + wl.Co, sizes[1] + wl.Ci
    head = header(dq, Co, Ci, wl.rank, fp8)
    opts = dict(kernel_product=dq.DQ_KERNEL_PRODUCT_FP8) if fp8 else {}
    whole = np.zeros(dq.dq_packed_weight_layout(wl.Co, wl.Ci, wl.rank).total_bytes, np.uint8)
    whole[:256] = head
    status, Y = run(dq, torch, case, whole, **opts)
    assert status == dq.DQ_ERR_BAD_PACKED_WEIGHT and (Y == -7).all()
    status, Y = run(dq, torch, case, head, **opts)   # 256 bytes of device memory, no more
    assert status == dq.DQ_ERR_BAD_PACKED_WEIGHT and (Y == -7).all()
