"""Calls whose tensors lie on several devices, or on another than the current
one, are refused before anything is launched.  The devices are pretended: CPU
tensors that say they are elsewhere, and a library that must not be called."""
import pytest

torch = pytest.importorskip("torch")


class On(torch.Tensor):
    """A tensor that says it lies on a GPU."""
    at = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.at)

    def get_device(self):
        return self.at


def on(index, t):
    t = t.as_subclass(On)
    t.at = index
    return t


class Untouched:
    """Sizes are asked of the library, nothing else."""

    def __getattr__(self, name):
        assert name.endswith("_bytes"), f"{name} was called"
        return lambda *sizes: 256


@pytest.fixture
def q(monkeypatch):
    import vector_codebook_codec_amd as pkg
    from vector_codebook_codec_amd import _lib

    monkeypatch.setattr(_lib, "load", Untouched)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return pkg


ADAPTERS = dict(X=torch.zeros(5, 64), codes=torch.zeros(40, 32, dtype=torch.uint8), scales=torch.zeros(40, 16, dtype=torch.uint8),
                A=torch.zeros(2, 4, 64), B=torch.zeros(2, 40, 4), index=torch.zeros(5, dtype=torch.int32), factors=torch.zeros(2),
                out=torch.zeros(5, 40), workspace=torch.zeros(256, dtype=torch.uint8))
ATTENTION = dict(Q=torch.zeros(5, 8, 64), codes=torch.zeros(2, 3, 2, 16, 32, dtype=torch.uint8),
                 scales=torch.zeros(2, 3, 2, 16, 2, dtype=torch.uint8), table=torch.zeros(5, 1, dtype=torch.int32),
                 lengths=torch.zeros(5, dtype=torch.int32), out=torch.zeros(5, 8, 64), lse=torch.zeros(5, 8),
                 workspace=torch.zeros(256, dtype=torch.uint8))


@pytest.mark.parametrize("name,tensors", [("qamw_mxfp4_adapter_matmul", ADAPTERS), ("qamw_mxfp4_cache_attention", ATTENTION)])
def test_refused(q, name, tensors):
    call = getattr(q, name)
    for there in tensors:
        with pytest.raises(ValueError, match="device"):
            call(**{k: on(int(k == there), t) for k, t in tensors.items()})
    with pytest.raises(ValueError, match="device"):
        call(**{k: on(1, t) for k, t in tensors.items()})
    with pytest.raises(AssertionError, match=name):              # and on one device, the current one, it is called
        call(**{k: on(0, t) for k, t in tensors.items()})
