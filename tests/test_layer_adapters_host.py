"""What adapter_forward would refuse, moe_forward refuses before the layer is enqueued: afterwards
`out` would hold the layer without its adapters. Host checks, no GPU."""
import pytest
import torch

import precision_moe_amd as pm

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
T, H, E, K, n, R = 4, 64, 4, 2, 3, 8


def _aligned(nbytes, shift=0):
    """uint8 memory that begins `shift` bytes behind a multiple of 256."""
    raw = torch.zeros(nbytes + 512 + shift, dtype=U8)
    at = -raw.data_ptr() % 256 + shift
    return raw[at:at + nbytes]


def _as(raw, dtype, *shape):
    return raw[:torch.Size(shape).numel() * dtype.itemsize].view(dtype).view(shape)


@pytest.fixture
def args():
    return dict(x=_as(_aligned(2 * T * H), BF, T, H), out=_as(_aligned(2 * T * H), BF, T, H),
                down=_as(_aligned(2 * n * R * H), BF, n, R, H), up=_as(_aligned(2 * n * R * H), BF, n, H, R),
                scale=_as(_aligned(4 * n), torch.float32, n), ids=_as(_aligned(4 * T), I32, T),
                ws=_aligned(pm.adapter_workspace_bytes(T, n, H, H, R)))


def _refused(args, match, workspace=None):
    P = pm.PreparedWeights(E, H, H, H, *([None] * 6))
    with pytest.raises(ValueError, match=match):
        pm.moe_forward(args["x"], torch.zeros(T, K, dtype=I32), torch.zeros(T, K), P, out=args["out"],
                       adapters=(args["down"], args["up"], args["scale"]), adapter_ids=args["ids"],
                       adapter_workspace=args["ws"], workspace=workspace)


@pytest.mark.parametrize("name", ["x", "down", "up", "scale", "ids"])
def test_out_over_what_the_adapters_read(args, name):
    big = _aligned(2 * n * R * H)
    args["out"] = _as(big, BF, T, H)
    t = args[name]
    args[name] = _as(big, t.dtype, *t.shape)
    _refused(args, f"out overlaps {name}|out overlaps adapter_{name}")


@pytest.mark.parametrize("name", ["x", "down", "up", "scale", "ids", "out"])
def test_workspace_over_an_argument(args, name):
    t = args[name]
    args[name] = _as(args["ws"], t.dtype, *t.shape)
    _refused(args, "overlaps")


@pytest.mark.parametrize("name", ["down", "up", "scale", "ids"])
def test_layer_workspace_over_what_the_adapters_read(args, name):
    ws = _aligned(pm.moe_workspace_bytes(T, K, E, H, H, pm.ACT_RELU2))
    t = args[name]
    args[name] = _as(ws[256:], t.dtype, *t.shape)
    _refused(args, "workspace overlaps", workspace=ws)


@pytest.mark.parametrize("name", ["down", "up", "ws"])
def test_alignment(args, name):
    t = args[name]
    raw = _aligned(t.numel() * t.element_size() + 16, shift=8)
    args[name] = raw if name == "ws" else _as(raw, t.dtype, *t.shape)
    _refused(args, "aligned")


@pytest.mark.parametrize("name", ["out", "ws"])
def test_devices(args, name):
    args[name] = args[name].to("meta")
    _refused(args, "on the device of x")
