"""The mixers' binding and devices (no GPU): tensors on a device that is not the current one, and workspaces or
status words on another device than the rest, are refused before the library is called (which would
launch on the current device, with the other one's addresses)."""
import pytest
import torch

from gated_delta_rule_36_gb300 import binding as kb

D = 128


class On0(torch.Tensor):
    def get_device(self):
        return 0


class On1(torch.Tensor):
    def get_device(self):
        return 1


class Library:
    """Stands for the loaded library: no call may reach it."""

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 256
        raise AssertionError(f"{name} was called")


@pytest.fixture(autouse=True)
def two_devices(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(kb, "_lib", Library())


def tensors(kind, *shapes, dtype=torch.bfloat16):
    return [torch.zeros(s, dtype=dtype).as_subclass(kind) for s in shapes]


def ws(kind):
    return tensors(kind, 1 << 10, dtype=torch.uint8)[0]


def calls(kind, workspace, status):
    t, b = tensors(kind, (4, 2, D))[0], tensors(kind, (1, 4, 2, D))[0]
    ld = tensors(kind, (2,), dtype=torch.float32)[0]
    return {
        "rope": lambda: kb.kda_qk_norm_rope(t, None, None, None, None, None, t, None, status=status, stream=0),
        "attn": lambda: kb.kda_attn_fwd(t, t, t, 1.0, t, workspace=workspace, stream=0),
        "lin": lambda: kb.kda_lin_fwd(b, b, b, ld, 1.0, b, workspace=workspace, stream=0),
        "step": lambda: kb.kda_lin_decode(t, t, t, ld, 1.0, t, stream=0),
    }


@pytest.mark.parametrize("name", ["rope", "attn", "lin", "step"])
def test_tensors_on_a_device_that_is_not_current(name):
    with pytest.raises(ValueError, match="current device"):
        calls(On1, ws(On1), ws(On1))[name]()


@pytest.mark.parametrize("name", ["rope", "attn", "lin"])
def test_workspaces_and_status_words_on_another_device(name):
    with pytest.raises(ValueError, match="other tensors' device"):
        calls(On0, ws(On1), ws(On1))[name]()
    with pytest.raises(ValueError, match="other tensors' device"):
        calls(On0, ws(torch.Tensor), "no tensor")[name]()


@pytest.mark.parametrize("name", ["rope", "attn", "lin", "step"])
def test_one_device_reaches_the_library(name):
    with pytest.raises(AssertionError, match="was called"):
        calls(On0, ws(On0), ws(On0))[name]()


def test_missing_keys_are_the_library_s_refusal(monkeypatch):
    monkeypatch.setattr(kb, "_lib", None)
    t = tensors(On0, (4, 2, D))[0]
    for workspace in (None, ws(On0)):
        monkeypatch.setattr(kb, "_workspace", lambda *a: ws(On0))
        with pytest.raises(kb.KDAError, match="k: missing"):
            kb.kda_attn_fwd(t, None, t, 1.0, t, workspace=workspace, stream=0)
