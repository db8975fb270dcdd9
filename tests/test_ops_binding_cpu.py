"""What the torch helpers around token IDs refuse before the library is called,
without a GPU: stand-ins for tensors, whose addresses nothing uses."""
import types

import pytest

from exact_bpe_tokenization_gb300 import binding as tt

torch = pytest.importorskip("torch")


class Standin:
    """As much of a tensor as the helpers look at."""
    def __init__(self, *shape, dtype=torch.float32, on=0, stride=None):
        self.shape, self.dtype, self.on = shape, dtype, on
        whole = [1]
        for n in shape[:0:-1]:
            whole.insert(0, whole[0] * n)
        self._stride = tuple(stride or whole)
        self._contiguous = self._stride == tuple(whole)

    device = property(lambda s: torch.device("cpu" if s.on < 0 else "cuda:%d" % s.on))
    is_cuda = property(lambda s: s.on >= 0)

    def get_device(self):
        return self.on

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._stride

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def element_size(self):
        return 1


class Library:
    """Counts the calls that reach it."""
    def __init__(self):
        self.calls = 0

    def tt_embed_grad_workspace(self, *_):
        return 1024

    def __getattr__(self, name):
        def call(*_):
            self.calls += 1
            return tt.TT_OK
        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    tt._load_torch()
    monkeypatch.setattr(tt, "lib", lambda: L)
    names = ("float32", "float16", "bfloat16", "int32", "int64", "uint8")
    monkeypatch.setattr(tt, "_torch", types.SimpleNamespace(
        empty=lambda shape, dtype, device: Standin(*(shape if isinstance(shape, tuple) else (shape,)), dtype=dtype, on=device.index),
        _C=types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda d: 0),
        **{n: getattr(torch, n) for n in names}))
    return L


def ints(n, dtype=torch.int32):
    return Standin(n, dtype=dtype)


CALLS = {
    "embed": (tt.embed, lambda: dict(ids=ints(4), table=Standin(300, 16), n_ids=ints(1, torch.int64), out=Standin(4, 16),
                                     status=ints(1))),
    "embed_grad": (tt.embed_grad, lambda: dict(ids=ints(4), dout=Standin(4, 16), n_vocab=300, n_ids=ints(1, torch.int64),
                                               out=Standin(300, 16), workspace=Standin(1024, dtype=torch.uint8),
                                               status=ints(1))),
    "token_loss": (tt.token_loss, lambda: dict(logits=Standin(4, 300), targets=ints(4), row_grads=Standin(4),
                                               dlogits=Standin(4, 300), status=ints(1))),
    "token_loss_grad": (tt.token_loss_grad, lambda: dict(logits=Standin(4, 300), targets=ints(4), lse=Standin(4),
                                                         row_grads=Standin(4), dlogits=Standin(4, 300), status=ints(1))),
    "sample": (tt.sample, lambda: dict(logits=Standin(4, 300), uniform=Standin(4), temperature=Standin(4), top_k=ints(4),
                                       top_p=Standin(4), min_p=Standin(4), status=ints(1))),
}
TENSORS = [(call, key) for call, (_, args) in CALLS.items() for key, v in args().items() if isinstance(v, Standin)]


@pytest.mark.parametrize("call", CALLS)
def test_what_fits_reaches_the_library(library, call):
    f, args = CALLS[call]
    f(**args())
    assert library.calls == 1


@pytest.mark.parametrize("call,key", TENSORS)
@pytest.mark.parametrize("on", [-1, 1])
def test_every_tensor_lies_on_one_device(library, call, key, on):
    """On another GPU, or in host memory, an address means something else."""
    f, args = CALLS[call]
    a = args()
    a[key].on = on
    with pytest.raises(ValueError):
        f(**a)
    assert library.calls == 0


@pytest.mark.parametrize("call", CALLS)
def test_the_tensors_device_is_the_current_one(library, call):
    f, args = CALLS[call]
    a = args()
    for v in a.values():
        if isinstance(v, Standin):
            v.on = 1
    with pytest.raises(ValueError, match="current device"):
        f(**a)
    assert library.calls == 0


@pytest.mark.parametrize("workspace", [Standin(1 << 20, dtype=torch.uint8, stride=(0,)), Standin(64, 64, stride=(128, 1)),
                                       Standin(1024, dtype=torch.uint8, on=-1), torch.empty(1024, dtype=torch.uint8)])
def test_a_workspace_holds_what_it_says(library, workspace):
    """More elements than bytes behind them (an expanded tensor), gaps, or host memory."""
    f, args = CALLS["embed_grad"]
    with pytest.raises(ValueError, match="workspace"):
        f(**{**args(), "workspace": workspace})
    assert library.calls == 0
