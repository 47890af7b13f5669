"""The 4-bit calls' Python entry points take tensors of one GPU, the current one (no GPU: stand-ins for
tensors; the library is replaced by a recorder)."""

import pytest
import torch

from hashed_gram_embedding_gb300 import _lib

BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


class Stand:
    """As much of a contiguous tensor as the checks read."""

    def __init__(self, dtype, *shape, device=1):
        self._t, self._device = torch.empty(shape, dtype=dtype), device
        self.dtype, self.shape = dtype, self._t.shape

    def get_device(self):
        return self._device

    @property
    def is_cuda(self):
        return self._device >= 0

    @property
    def device(self):
        return f"device {self._device}"

    def on(self, device):
        self._device = device
        return self

    def data_ptr(self):
        return 256

    def __getattr__(self, name):
        if name in ("stride", "dim", "numel", "is_contiguous"):
            return getattr(self._t, name)
        raise AttributeError(name)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


class Stream:
    cuda_stream = 0


@pytest.fixture
def library(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(_lib, "lib", lambda: recorder)
    monkeypatch.setattr(_lib, "_one_gpu", False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    return recorder


def cache():
    return dict(cache=Stand(U8, 4, 2, 1, 16 * 136), block_table=Stand(I32, 1, 4), query_start_loc=Stand(I32, 2),
                kv_lens=Stand(I32, 1))


def calls():
    return {
        "ple_kv_append": dict(q=Stand(BF16, 3, 4, 128), k=Stand(BF16, 3, 2, 128), v=Stand(BF16, 3, 2, 128),
                              cos_sin=Stand(F32, 9, 64), q_out=Stand(BF16, 3, 4, 128), positions=Stand(I32, 3),
                              dev_err=Stand(I32, 1), **cache()),
        "ple_kv_read": dict(k_out=Stand(BF16, 3, 2, 128), v_out=Stand(BF16, 3, 2, 128), dev_err=Stand(I32, 1), **cache()),
        "ple_kv_attention": dict(q=Stand(BF16, 3, 4, 128), out=Stand(BF16, 3, 4, 128), workspace=Stand(U8, 512),
                                 dev_err=Stand(I32, 1), **cache()),
        "ple_proj_w4": dict(x=Stand(BF16, 3, 256), codes=Stand(U8, 8, 128), scales=Stand(BF16, 8, 2),
                            out=Stand(BF16, 3, 8), zeros=Stand(U8, 8, 2), dev_err=Stand(I32, 1)),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_one_device(library, name):
    entry = getattr(_lib, name)
    entry(**calls()[name], stream=Stream())
    assert library.calls == [name]
    for argument in calls()[name]:
        for device in (-1, 0, 2):
            args = calls()[name]
            args[argument].on(device)
            with pytest.raises(ValueError):
                entry(**args, stream=Stream())
    for device in (-1, 0):  # all together, but not on the current one
        with pytest.raises(ValueError):
            entry(**{k: t.on(device) for k, t in calls()[name].items()}, stream=Stream())
    assert library.calls == [name]


@pytest.mark.parametrize("name", list(calls()))
def test_the_error_word(library, name):
    entry = getattr(_lib, name)
    for word in (Stand(torch.int64, 1), Stand(I32, 0), Stand(F32, 1)):
        with pytest.raises(ValueError):
            entry(**dict(calls()[name], dev_err=word), stream=Stream())
    entry(**dict(calls()[name], dev_err=None), stream=Stream())
    assert library.calls == [name]


def test_one_gpu_is_asked_for_once(library, monkeypatch):
    asked = []
    monkeypatch.setattr(_lib, "_one_gpu", None)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: asked.append(1) or 1)
    for name in calls():
        getattr(_lib, name)(**calls()[name], stream=Stream())
    assert len(asked) == 1 and library.calls == list(calls())
    for name, first in (("ple_kv_append", "k"), ("ple_kv_read", "v_out"), ("ple_kv_attention", "q"), ("ple_proj_w4", "x")):
        args = calls()[name]
        args[first].on(-1)
        with pytest.raises(ValueError):
            getattr(_lib, name)(**args, stream=Stream())


def test_no_tokens_in_tensors_of_any_strides(library):
    """An empty tensor's strides say nothing (NumPy's and a slice's differ from a fresh tensor's)."""
    def empty(*shape):
        t = Stand(BF16, *shape)
        t._t = torch.empty_strided(shape, tuple(range(1, len(shape) + 1)), dtype=BF16)
        return t

    _lib.ple_kv_append(empty(0, 4, 128), empty(0, 2, 128), empty(0, 2, 128), None, **cache(), q_out=empty(0, 4, 128),
                       stream=Stream())
    _lib.ple_kv_attention(empty(0, 4, 128), **cache(), out=empty(0, 4, 128), workspace=Stand(U8, 512), stream=Stream())
    _lib.ple_proj_w4(empty(0, 256), Stand(U8, 8, 128), Stand(BF16, 8, 2), Stand(BF16, 0, 8), stream=Stream())
    assert library.calls == ["ple_kv_append", "ple_kv_attention", "ple_proj_w4"]
    with pytest.raises(ValueError):
        _lib.ple_kv_append(empty(0, 4, 128), empty(0, 2, 128), empty(0, 2, 64), None, **cache(), q_out=empty(0, 4, 128),
                           stream=Stream())
