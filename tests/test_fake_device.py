"""What calls of the group norm and the rotary positions would launch where
there is a device, seen without one (tests/_fake_device.py)."""

import ctypes
import inspect

import pytest
import torch

import _fake_device
import conftest
import test_blocks_abi as abi


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return _fake_device.load(tmp_path_factory.mktemp("fake"))


def refusals():
    """(name, call, arguments, status) of every host-side refusal in test_blocks_abi."""
    for fn, call in ((abi.test_gn_fwd_rejects_on_host, abi.gn_fwd),
                     (abi.test_gn_bwd_rejects_on_host, abi.gn_bwd),
                     (abi.test_rope_fwd_rejects_on_host, abi.rope),
                     (abi.test_rope_bwd_rejects_on_host, abi.rope_b)):
        (mark,) = [m for m in fn.pytestmark if m.name == "parametrize"]
        for i, (kw, want) in enumerate(mark.args[1]):
            yield pytest.param(call, kw, want, id=f"{fn.__name__}-{i}")


@pytest.mark.parametrize("call,kw,want", list(refusals()))
def test_refusals_come_before_any_launch(lib, call, kw, want):
    """With a device, too: their addresses are made up."""
    _fake_device.reset(lib)
    assert call(lib, **kw) == want
    assert _fake_device.counts(lib)["launches"] == 0


class Item:
    """A collected test, as far as the hook looks at one."""

    def __init__(self, name):
        self.originalname, self.marks = name, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def test_accepted_calls_on_made_up_addresses_need_a_machine_without_gpu(lib, monkeypatch):
    """The unmarked tests that go through the C library without a refusal are
    those that would launch, and a visible GPU skips them."""
    launch = []
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    for name, fn in inspect.getmembers(abi, inspect.isfunction):
        if not name.startswith("test_") or list(inspect.signature(fn).parameters) != ["lib"]:
            continue
        _fake_device.reset(lib)
        try:
            fn(lib)
        except AssertionError:
            pass        # it expects to end at the missing device
        if _fake_device.counts(lib)["launches"]:
            launch.append(name)
    assert launch == ["test_gn_fwd_slices_of_one_buffer", "test_rope_overlap_of_packed_heads"]
    items = [Item(n) for n in launch + ["test_gn_fwd_rejects_on_host"]]
    conftest.pytest_collection_modifyitems(items)
    assert not any(i.marks for i in items)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    items = [Item(n) for n in launch + ["test_gn_fwd_rejects_on_host"]]
    conftest.pytest_collection_modifyitems(items)
    assert [i.marks for i in items] == [["skip"], ["skip"], []]


def test_many_samples_without_gradients_of_their_parameters(lib):
    """The limit of 65535 samples is that of the gradients' sums."""
    many = dict(ps=64, N=70000, rows=1, xs=0, ds=0, os_=64, wb=1 << 30)
    # the statistics and the workspace would lie in one another
    far = dict(m=1 << 48, r=1 << 49, ws=1 << 50, dg=None, db=None)
    _fake_device.reset(lib)
    assert abi.gn_bwd(lib, **many, **far) == abi.OK
    counts = _fake_device.counts(lib)
    assert counts["launches"] > 0 and counts["finalizes"] == 0
    _fake_device.reset(lib)
    for grad in ("dg", "db"):
        assert abi.gn_bwd(lib, **many, **{**far, grad: 1 << 51}) == abi.SHAPE
    assert _fake_device.counts(lib)["launches"] == 0


@pytest.mark.parametrize("most", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("sms", [1, 8, 40, 152])
def test_clusters_no_larger_than_the_device_places(lib, most, sms):
    """Every forward runs, in smaller clusters or in two launches, with the
    workspace that the query gives for that device."""
    _fake_device.reset(lib, sms, most)
    need, seen = ctypes.c_size_t(), set()
    for N, rows, C, groups in ((1, 40, 64, 8), (2, 4096, 320, 32), (16, 1024, 1280, 32),
                               (1, 7, 8, 1), (4, 205, 192, 32), (2, 262144, 256, 32),
                               (3, 2867, 165, 5), (1, 100000, 8, 8), (200, 3, 2048, 1)):
        assert lib.gn_workspace_bytes(N, rows, C, groups, abi.BF16, 0, ctypes.byref(need)) == abi.OK
        _fake_device.reset(lib, sms, most)
        far = dict(x=1 << 45, y=1 << 46, m=1 << 47, r=1 << 48, ws=1 << 49)
        assert abi.gn_fwd(lib, N=N, rows=rows, C=C, groups=groups, xs=rows * C, xr=C, ys=rows * C,
                          yr=C, wb=need.value, **far) == abi.OK, (N, rows, C)
        got = _fake_device.counts(lib)
        assert got["launches"] >= 1 and got["cluster"] <= most
        seen.add(got["cluster"])
    assert sms < 152 or most in seen
