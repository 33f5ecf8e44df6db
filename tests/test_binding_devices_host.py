"""The binding's training calls take every tensor on the current device, the caller's
workspace included.  Host memory in tensors that claim to be on a device: nothing is
launched without a GPU."""

import pytest
import torch

from bitlinear_bl_forward_b200 import bl

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="tensors that only claim to be on a device")


class On(torch.Tensor):
    """A tensor that says it is on device `dev`."""
    dev = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.dev


def on(dev, *shape, dtype=torch.bfloat16):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.dev = dev
    return t


M, K, N = 6, 64, 12


def calls(ws):
    x, dy = on(0, M, K), on(0, M, N)
    q, s = on(0, M, K, dtype=torch.int8), on(0, M, dtype=torch.float32)
    wp, g = on(0, N, K // 4, dtype=torch.uint8), on(0, 1, dtype=torch.float32)
    return {
        "forward_checkpoint": lambda: bl.bl_forward_checkpoint(x, wp, g, N, workspace=ws),
        "backward_input": lambda: bl.bl_backward_input(dy, wp, g, K, workspace=ws),
        "backward_weight": lambda: bl.bl_backward_weight(dy, q, s, workspace=ws),
        "norm_backward": lambda: bl.bl_norm_backward(x, x, bl.BL_NORM_RMS, s, weight=on(0, K), workspace=ws,
                                                     dweight=on(0, K, dtype=torch.float32)),
    }


@pytest.mark.parametrize("name", ["forward_checkpoint", "backward_input", "backward_weight", "norm_backward"])
def test_a_workspace_on_another_device_is_refused(name, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bl, "_raw_stream", lambda dev: 0)
    # on the current device the call gets as far as the launch, which there is no GPU for
    with pytest.raises(bl.BLError) as e:
        calls(on(0, 1 << 20, dtype=torch.uint8))[name]()
    assert e.value.status == 5
    with pytest.raises(ValueError, match="workspace"):
        calls(on(1, 1 << 20, dtype=torch.uint8))[name]()
