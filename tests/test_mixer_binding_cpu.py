"""What the mixer binding does on the host before a call reaches the library (no GPU needed)."""
import types

import numpy as np
import pytest
import torch

from linear_attention_recurrent_gdn_gb300 import build


@pytest.fixture(scope="module")
def mx():
    build.build()
    from linear_attention_recurrent_gdn_gb300 import mixer
    return mixer


# ------------------------------------------------------------------ devices --
class Devices:
    """Two devices on the host: which one is current, and what the library saw as it was called."""

    def __init__(self, mx, monkeypatch):
        self.current, self.seen, outer = 0, [], self

        class Guard:
            def __init__(self, dev):
                self.dev = dev

            def __enter__(self):
                self.before, outer.current = outer.current, self.dev

            def __exit__(self, *exc):
                outer.current = self.before

        monkeypatch.setattr(mx, "_device", lambda: self.current, raising=False)
        monkeypatch.setattr(mx, "_raw_stream", lambda dev: 1000 + dev)
        monkeypatch.setattr(torch.cuda, "device", Guard)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(
            device_index=self.current if device is None else device,
            cuda_stream=1000 + (self.current if device is None else device)))

    def library(self, result):
        def call(*args):
            self.seen.append((self.current,) + args)
            return result
        return call


def test_calls_run_with_their_tensors_device_current(mx, monkeypatch):
    """A launch goes to the current device whatever its stream; stream 0 is every device's default stream."""
    devs = Devices(mx, monkeypatch)
    mx._call(devs.library(0), b"args", 0)
    mx._call(devs.library(0), b"args", 1)
    assert [s[:3] for s in devs.seen] == [(0, b"args", 1000), (1, b"args", 1001)]
    assert devs.current == 0
    with pytest.raises(mx._dl.DeltaLogError):
        mx._call(devs.library(1), b"args", 1)
    assert devs.current == 0


def test_sync_reads_the_status_of_the_named_device(mx, monkeypatch):
    devs = Devices(mx, monkeypatch)
    monkeypatch.setattr(mx, "_lib", types.SimpleNamespace(dl_mixer_sync=devs.library(0)))
    mx.sync()
    mx.sync(1)
    assert [s[:2] for s in devs.seen] == [(0, 1000), (1, 1001)] and devs.current == 0


# --------------------------------------------------------------- host lists --
@pytest.mark.parametrize("given,dtype", [
    ([0.7, 1.0], np.int32), (np.array([0.0, 1.0]), np.int32), ([1, None], np.int32), (["0", "1"], np.int32),
    (np.array([1, 2 ** 32 + 1]), np.int32), ([2 ** 32 + 1, 0], np.int32), ([-2 ** 31 - 1, 0], np.int32),
    (np.array([3, 2 ** 31], dtype=np.uint32), np.int32), ([0, 2 ** 70], np.int32),
    ([0, 256], np.uint8), ([-1, 0], np.uint8), (np.array([0.5, 1.0]), np.uint8),
    ([0, 1, 2], np.int32), ([[0, 1]], np.int32), (5, np.int32),
])
def test_host_lists_that_are_refused(mx, given, dtype):
    """Slots, lengths and flags are whole numbers of their type; none is cut or wrapped to one."""
    with pytest.raises((ValueError, TypeError)):
        mx._host(given, dtype, 2, "list")


@pytest.mark.parametrize("given,dtype,want", [
    ([3, 2 ** 31 - 1], np.int32, [3, 2 ** 31 - 1]), (np.array([-1, 7]), np.int32, [-1, 7]),
    (np.array([1, 9, 2, 9], dtype=np.int32)[::2], np.int32, [1, 2]), (torch.tensor([4, 5]), np.int32, [4, 5]),
    (np.array([True, False]), np.uint8, [1, 0]), ([True, False], np.uint8, [1, 0]), ([1, 0], np.uint8, [1, 0]),
    (range(2), np.int32, [0, 1]),
])
def test_host_lists_that_are_taken(mx, given, dtype, want):
    a, at = mx._host(given, dtype, 2, "list")
    assert a.dtype == dtype and a.tolist() == want and at == a.ctypes.data and a.flags.c_contiguous


def test_empty_and_ready_lists(mx):
    assert mx._host([], np.int32, 0, "list")[0].shape == (0,)
    ready = np.array([1, 2], np.int32)
    assert mx._host(ready, np.int32, 2, "list")[0] is ready


# ------------------------------------------------------------- derivatives --
def test_tensors_that_are_differentiated_are_refused(mx):
    """Backward or forward: a result without its derivative would be taken for a constant."""
    fwd = torch.autograd.forward_ad
    t = torch.ones(3)
    check = lambda v: mx._check("weight", v, (3,), torch.float32, -1)  # noqa: E731  (a CPU tensor's device)
    check(t)
    with pytest.raises((ValueError, TypeError)):
        check(torch.ones(3, requires_grad=True))
    with torch.no_grad():
        check(torch.ones(3, requires_grad=True))
    with fwd.dual_level():
        check(t)
        with torch.inference_mode():
            check(torch.ones(3))
        with pytest.raises((ValueError, TypeError)):
            check(fwd.make_dual(t, torch.ones(3)))
    check(t)
    seen = []

    def f(v):
        seen.append(mx._differentiated(v))
        return v * 2
    torch.func.jvp(f, (t,), (torch.ones(3),))
    assert seen == [True]


# -------------------------------------------------------------------- names --
def test_unknown_activations_and_norms(mx):
    assert [mx._one_of(mx._ACT, a, "activation") for a in (None, "none", "silu", "sigmoid")] == [0, 0, 1, 2]
    for names, name in ((mx._ACT, "relu"), (mx._ACT, 1), (mx._KIND, None), (mx._KIND, ["rms"])):
        with pytest.raises(ValueError, match="expected one of"):
            mx._one_of(names, name, "name")
