"""The calls of beam selection and of the paged cache's upkeep on tensors of another device than the current one: the
extension leaves them to the Python wrapper, which makes the call again with the tensors' device current.  The current
device is stood in for, so that one GPU, or none, will do."""
import pytest
import torch

from exact_attention_staged_gb300 import api, build

CALLS = {"paged_reserve": 8, "paged_fork": 4, "paged_free": 4, "paged_compact": 4, "paged_copy": 6, "beam_select": 10}


class Current:
    """The current device: `answers`, one call after the other, the last one from then on."""

    def __init__(self):
        self.answers, self.asked = [0], 0

    def __call__(self):
        self.asked += 1
        return self.answers.pop(0) if len(self.answers) > 1 else self.answers[0]


@pytest.fixture
def current(monkeypatch):
    """The extension set up with another source of the current device, and as it was afterwards."""
    build.build()
    where = Current()
    with monkeypatch.context() as m:
        m.setattr(api, "_current_device", where)
        m.setattr(api, "_binding", None)
        api._calls()
        yield where
    api._binding = None
    api._calls()


class Tensor:
    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_left_to_the_wrapper(current, name):
    call, more = getattr(api._calls(), name), [None] * (CALLS[name] - 1)
    for here, there in ((0, 1), (1, 0), (3, 2)):
        current.answers = [here]
        assert call(Tensor(there), *more) is NotImplemented
        with pytest.raises(AttributeError):  # goes on to look at the tensor
            call(Tensor(here), *more)


def test_an_error_of_the_current_device_is_passed_on(current):
    def broken():
        raise RuntimeError("no device")
    api._current_device, api._binding = broken, None  # put back by the fixture
    for name, n in CALLS.items():
        with pytest.raises(RuntimeError, match="no device"):
            getattr(api._calls(), name)(Tensor(0), *[None] * (n - 1))


@pytest.mark.gpu
def test_calls_away_from_the_current_device_come_to_the_same(cuda_lib, current):
    dev = "cuda:0"

    def index(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def all_calls():
        x = torch.randn(2, 3, 700, generator=torch.Generator(device=dev).manual_seed(1), device=dev)
        table, refs, kv = index([[-1] * 4 for _ in range(3)]), index([0] * 40), index([20, 9, 1])
        k, v = (torch.randn(2, 40, 2, 8, 64, generator=torch.Generator(device=dev).manual_seed(i),
                            device=dev).half() for i in (2, 3))
        out = list(cuda_lib.beam_select(x, x[..., 0].contiguous()))
        cuda_lib.paged_reserve(table, kv, refs, 8, index([0, 20, 29, 30]), tokens=30)
        cuda_lib.paged_fork(table, index([0, 0, 1]), refs, kv)
        kv += 1
        copies = cuda_lib.paged_reserve(table, kv, refs, 8)
        cuda_lib.paged_copy(k, v, copies[0], copies[1], copies[2])
        cuda_lib.paged_free(table, index([0, 9, 10]), refs, 8)
        out += list(cuda_lib.paged_compact(table, refs, moves=index([[-1] * 20] * 2)))
        assert cuda_lib.sync_status() == 0
        return out + [copies, table, refs, kv, k, v]
    want = all_calls()
    before = current.asked
    current.answers = [1, 0] * 12  # each call: away, then with the device current
    got = all_calls()
    assert current.asked - before == 2 * 7
    assert all(torch.equal(a, b) for a, b in zip(got, want))
