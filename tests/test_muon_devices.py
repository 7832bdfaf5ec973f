"""Which linears one PoetxMuon takes: those whose parameters lie on one device, however that device was named."""

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import layer as L


def test_one_device_under_two_names():
    lays = [L.PoetxLinear(64, 48, 16, device="cpu") for _ in range(2)]
    for lay, name in zip(lays, ("cuda", "cuda:0")):  # what PoetxLinear keeps of device="cuda" and of device="cuda:0"
        lay.device = torch.device(name)
    opt = L.PoetxMuon(lays)
    assert opt.device == lays[0].q_R.device and opt.ws.device == opt.device


def test_two_devices_are_refused():
    with pytest.raises(ValueError, match="share a device"):
        L.PoetxMuon([L.PoetxLinear(64, 48, 16, device=d) for d in ("cpu", "meta")])


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_step_of_linears_under_two_names():
    lays = [L.PoetxLinear(64, 48, 16, device=d) for d in ("cuda", "cuda:0")]
    opt = L.PoetxMuon(lays, lr=0.1)
    g = torch.randn(lays[0].q_R.shape, device="cuda"), torch.randn(lays[0].q_P.shape, device="cuda")
    assert not opt.step([g, g])
    torch.cuda.synchronize()
    assert lays[0].q_R.any() and torch.equal(lays[0].q_R, lays[1].q_R) and torch.equal(lays[0].q_P, lays[1].q_P)
