"""Calls with a stream of their own, without a GPU: what a call allocates must
belong to the stream that its kernels run on."""
import inspect

import pytest
import torch

from depth_wise_attention_gb300 import attnres

CALLS = sorted(n for n, f in vars(attnres).items()
               if inspect.isfunction(f) and f.__module__ == attnres.__name__ and not n.startswith("_")
               and "stream" in inspect.signature(f).parameters and n != "attnres_sync_status")


class Stream:
    """A stream of a device, by its number."""
    device_type = 1

    def __init__(self, stream_id, device_index):
        self.stream_id, self.device_index = stream_id, device_index


class Entered(Exception):
    pass


def test_the_calls_are_found():
    assert len(CALLS) == 29 and "attnres_norm_bwd" in CALLS and "msar_block_phase1_bwd" in CALLS


def call(f, stream, by_name):
    parameters = inspect.signature(f).parameters
    if by_name:
        f(*[None] * sum(p.default is inspect.Parameter.empty for p in parameters.values()), stream=stream)
    else:
        f(*[None] * list(parameters).index("stream"), stream)


@pytest.mark.parametrize("by_name", [True, False])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_runs_under_its_stream(name, by_name, monkeypatch):
    """The given stream is the current one while the call runs (here: until it finds that its arguments are None),
    and the one before it is again afterwards, also when the call fails."""
    now = [(7, 0, 1)]

    def set_stream(stream_id, device_index, device_type):
        now.append((stream_id, device_index, device_type))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentStream", lambda dev: now[-1])
    monkeypatch.setattr(torch._C, "_cuda_setStream", set_stream)
    f = getattr(attnres, name)
    failures = (AttributeError, TypeError, ValueError, RuntimeError)
    with pytest.raises(failures):
        call(f, Stream(9, 0), by_name)
    assert now == [(7, 0, 1), (9, 0, 1), (7, 0, 1)]
    # none given, or the current one: nothing is switched
    for stream in (None, Stream(7, 0)):
        with pytest.raises(failures):
            call(f, stream, by_name)
    assert len(now) == 3


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device(name, monkeypatch):
    """Its device becomes the current one too."""
    mine, entered = Stream(9, 1), []

    class Context:
        def __init__(self, stream):
            entered.append(stream)

        def __enter__(self):
            raise Entered

        def __exit__(self, *a):
            return False
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    with pytest.raises(Entered):
        call(getattr(attnres, name), mine, True)
    assert entered == [mine]
