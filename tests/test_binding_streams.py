"""What the binding allocates for a call on a given stream comes from that stream's pool: memory of
another stream's could be handed out again, or still be in use there, while the call works on it.
Stand-ins for tensors, streams and the library, so that no GPU is needed."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

import block_sparse_attention_gather_b200 as bsa
from block_sparse_attention_gather_b200 import _native

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class FakeTensor(torch.Tensor):
    """A CPU tensor that says it is on the first GPU."""

    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_subclass(cls, t)

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x1000

    def record_stream(self, stream):
        self.used_on = stream


class FakeLib:
    """Every call succeeds; sizes are 4096 bytes."""

    def __getattr__(self, name):
        return lambda *a: 4096 if "size" in name else 0


MAIN, SIDE = SimpleNamespace(cuda_stream=0x1000), SimpleNamespace(cuda_stream=0x2000)


@pytest.fixture
def made(monkeypatch):
    """The tensors allocated on the device, with the stream that was current as made_on."""
    current, seen = [MAIN], []
    empty = torch.empty

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def record(*size, device=None, **kw):
        if device is None or torch.device(device).type == "cpu":
            return empty(*size, **kw)
        t = FakeTensor(empty(*size, **kw))
        t.made_on, t.used_on = current[-1], None
        seen.append(t)
        return t

    def like(t):
        return record(t.shape, dtype=t.dtype, device=t.device)

    monkeypatch.setattr(torch, "empty", record)
    monkeypatch.setattr(torch, "empty_like", like)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(_native, "lib", FakeLib)
    return seen


def rows(n, dtype=BF):
    return FakeTensor(torch.zeros(2, n, 128, dtype=dtype))


def ints(*v):
    return FakeTensor(torch.tensor(v, dtype=I32))


def perms(n):
    p = FakeTensor(torch.zeros(2, n, dtype=I32))
    return p, p, ints(0, n), ints(0, n)


def host(n):
    x, p, o = torch.zeros(2, n, 128, dtype=BF), torch.zeros(2, n, dtype=I32), torch.tensor([0, n])
    return x, x, x, p, p, o.int(), o.int()


CALLS = {
    "attend_dense": (3, lambda s: bsa.spark_attend_dense(rows(5), rows(9), rows(9), stream=s)),
    "qk_norm_rope": (3, lambda s: bsa.spark_qk_norm_rope(rows(5), rows(5), rows(5), stream=s)),
    "attend_ranges": (1, lambda s: bsa.spark_attend_ranges(5, ints(0, 5), stream=s)),
    "forward_joint": (3, lambda s: bsa.spark_bsa_forward_joint(
        rows(9), rows(9), rows(9), rows(4), rows(4), rows(4), *perms(9), 0.5, stream=s)),
    "reblock": (4, lambda s: bsa.spark_reblock(rows(9), rows(9), 4, stream=s)),
    "forward_host": (2, lambda s: bsa.spark_bsa_forward_host(
        *host(9), 0.5, out=host(9)[0], streams=(s, MAIN, MAIN))),
}


def test_streams_of_the_host_pipeline_may_be_any_iterable(made):
    bsa.spark_bsa_forward_host(*host(9), 0.5, out=host(9)[0], streams=iter([SIDE, MAIN, MAIN]))
    assert [t.made_on for t in made] == [SIDE] * 2


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_given_is_no_other_stream(made, name, monkeypatch):
    def switched(stream):
        raise AssertionError("switched streams")

    monkeypatch.setattr(torch.cuda, "stream", switched)
    CALLS[name][1](MAIN)
    assert all(t.used_on is None for t in made) and len(made) == CALLS[name][0]


@pytest.mark.parametrize("name", CALLS)
def test_allocations_come_from_the_stream_of_the_call(made, name):
    count, call = CALLS[name]
    call(SIDE)
    assert [t.made_on for t in made] == [SIDE] * count
    assert [t.used_on for t in made] == [MAIN] * count       # where the caller may drop them
